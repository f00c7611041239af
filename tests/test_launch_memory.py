"""Shared memory of launches and of early ends (CPU, from the source). What a kernel that moves its base up to the
next 1024 bytes is launched with, and opted in for, has to hold its layout behind the largest move, or its
barriers lie behind the allocation wherever the base is not aligned by itself."""
import os
import re

from bit_block_scaled_nvfp4_b200 import build

CSRC = os.path.join(build.HERE, "csrc")
MOVED = re.compile(r"smem_raw \+ \(\(1024u - \(smem_u32\(smem_raw\) & 1023u\)\) & 1023u\)"
                   r"|\(reinterpret_cast<uintptr_t>\(smem_raw\) \+ 1023\) & ~")


def _source(name):
    return open(os.path.join(CSRC, name)).read()


def _moving_kernels():
    names = set()
    for f in os.listdir(CSRC):
        for body in _source(f).split("__global__")[1:]:
            head = re.search(r"\b(\w+_kernel)\s*\(", body)
            if head and MOVED.search(body):
                names.add(head.group(1))
    return names


def test_kernels_that_align_their_base_are_launched_with_the_room_for_it():
    names = _moving_kernels()
    assert names >= {"attn_fwd_kernel", "attn_pp_kernel", "decode_kernel"}
    text = _source("qk4v8.cu")
    for name in sorted(names):
        launches = re.findall(rf"\b{name}<[^;]*?><<<([^;]*?)>>>", text)
        opt_ins = re.findall(rf"set_smem\({name}<[^;]*?>, ([^;]*?)\)", text)
        assert launches and opt_ins, name
        for sizes in launches:
            assert "SMEM_ALLOC" in sizes and "SMEM_BYTES" not in sizes, f"{name}<<<{sizes}>>>"
        for size in opt_ins:
            assert "SMEM_ALLOC" in size, f"{name}: opted in for {size}"


def test_the_room_holds_the_largest_move():
    for f in ("attn_fwd.cuh", "attn_pp.cuh", "decode.cuh"):
        assert re.search(r"SMEM_ALLOC = SMEM_BYTES \+ 1024;", _source(f)), f


def test_no_role_of_the_prompt_kernel_leaves_copies_on_their_way():
    """A wait that gives up ends a role early: the decoding warps' copies into shared memory, and Q's, are waited
    for behind their loops, whichever way these end."""
    text = _source("kv4_prompt.cuh")
    text = text[text.index("void __launch_bounds__(512, 1)"):]
    queries, rest = text.split("K and V decoding", 1)
    decoding = rest.split("= softmax =", 1)[0]
    assert queries.rindex("mbar_wait(kConvertQ ? q_raw : q_full") > queries.rindex("tma_load_3d(")
    assert "cp_async_wait<0>()" in decoding and decoding.rindex("cp_async_wait<0>()") > decoding.rindex("cp_async_commit()")
