"""Host-side checks of the 4-bit cache's calls, without a GPU: the binding checks every buffer
against the sizes it passes on, the library rejects bad arguments before touching the device, and
the oracle's cache, attention and page pool agree with direct computations."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from bit_block_scaled_nvfp4_b200 import _lib, api, build, paged
from oracle import kv4 as OK
from oracle.formats import e2m1_decode, e4m3_decode

DEVICE_ERR = "tensors on one CUDA device"
FAKE = 1 << 20          # aligned fake device addresses: never dereferenced on these paths
BAD, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def cache(pages=40, hkv=2, d=128):
    return paged.empty_cache4(pages, hkv, d, 0.0625, 0.0625, "cpu")


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


# ---- the binding ----
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_token_calls_accept_producer_shapes(dtype):
    wide = torch.empty(9, 5, 128, dtype=dtype)
    for k in (torch.empty(9, 2, 128, dtype=dtype), wide[:, 1:3], torch.empty(0, 2, 128, dtype=dtype), wide[3:4, :2]):
        with pytest.raises(ValueError, match=DEVICE_ERR):
            api.kv4_append_paged(cache(), k, k, i32(4), i32(3), i32(3, 8))
    with pytest.raises(ValueError, match=DEVICE_ERR):
        api.kv4_read_paged(cache(), i32(4), i32(3), i32(3, 8), 9, dtype=torch.float32)


def test_token_calls_refuse_other_buffers():
    k = torch.empty(9, 2, 128, dtype=torch.bfloat16)
    args = (i32(4), i32(3), i32(3, 8))
    with pytest.raises(TypeError):
        api.kv4_append_paged(cache(), k.float(), k.float(), *args)
    with pytest.raises(TypeError, match="v"):
        api.kv4_append_paged(cache(), k, k.half(), *args)
    with pytest.raises(ValueError, match="v"):
        api.kv4_append_paged(cache(), k, k[:8], *args)
    with pytest.raises(ValueError, match="k"):
        api.kv4_append_paged(cache(hkv=3), k, k, *args)
    with pytest.raises(ValueError, match="cu"):
        api.kv4_append_paged(cache(), k, k, i32(3), i32(3), i32(3, 8))
    with pytest.raises(ValueError, match="start"):
        api.kv4_append_paged(cache(), k, k, i32(4), i32(2), i32(3, 8))
    with pytest.raises(TypeError, match="page_table"):
        api.kv4_append_paged(cache(), k, k, i32(4), i32(3), i32(3, 8).long())
    for bad in (torch.empty(9, 128, 2, dtype=k.dtype).transpose(1, 2),     # channels apart
                torch.empty(9, 4, 128, dtype=k.dtype)[:, ::2],             # heads apart
                torch.empty(2, 128, dtype=k.dtype).expand(9, 2, 128),      # one token for all
                torch.empty(9, 260, dtype=k.dtype)[:, :256].unflatten(1, (2, 128))):   # tokens 4 elements off
        with pytest.raises(ValueError, match="tokens"):
            api.kv4_append_paged(cache(), bad, k, *args)
    other = cache()
    other.v_scales = other.v_scales[:, :, :4].contiguous()
    with pytest.raises(ValueError, match="cache.v_scales"):
        api.kv4_append_paged(other, k, k, *args)
    other = cache()
    other.k_tensor_scale = torch.zeros(2)
    with pytest.raises(ValueError, match="cache.k_tensor_scale"):
        api.kv4_append_paged(other, k, k, *args)
    with pytest.raises(TypeError, match="fp32"):
        api.kv4_read_paged(cache(), *args, 9, dtype=torch.float64)
    with pytest.raises(ValueError, match="out"):
        api.kv4_read_paged(cache(), *args, 9, out=(k[:8], k[:8]))


def test_attention_checks_its_buffers():
    q, t, c = torch.empty(6, 8, 128, dtype=torch.float16), i32(3, 8), i32(3)
    for ok in (q, torch.empty(6, 12, 128, dtype=torch.float16)[:, 2:10]):
        with pytest.raises(ValueError, match=DEVICE_ERR):
            api.attn_kv4_paged(ok, cache(), t, c, 500, cu_q=i32(4), max_q=4)
    with pytest.raises(ValueError, match="one token per sequence"):
        api.attn_kv4_paged(q, cache(), t, c, 500)
    with pytest.raises(ValueError, match="one token per sequence"):
        api.attn_kv4_paged(q[:3], cache(), t, c, 500, max_q=2)
    with pytest.raises(TypeError):
        api.attn_kv4_paged(q.float(), cache(), t, c, 500, cu_q=i32(4), max_q=4)
    with pytest.raises(ValueError, match="q"):
        api.attn_kv4_paged(q[..., :64], cache(), t, c, 500, cu_q=i32(4), max_q=4)
    with pytest.raises(ValueError, match="context_lens"):
        api.attn_kv4_paged(q, cache(), t, i32(4), 500, cu_q=i32(4), max_q=4)
    with pytest.raises(ValueError, match="out"):
        api.attn_kv4_paged(q, cache(), t, c, 500, cu_q=i32(4), max_q=4, out=q[:5])
    with pytest.raises(TypeError, match="out"):
        api.attn_kv4_paged(q, cache(), t, c, 500, cu_q=i32(4), max_q=4, out=q.bfloat16())
    with pytest.raises(ValueError, match="cu_q"):
        api.attn_kv4_paged(q, cache(), t, c, 500, cu_q=i32(3), max_q=4)
    with pytest.raises(ValueError, match=DEVICE_ERR):
        api.KV4AttentionPlan(cache(), t, c, 500, 8)


def test_pool_calls_check_their_buffers():
    pool, t, lens = paged.empty_pool(40, "cpu"), i32(3, 8), i32(3)
    for call in (lambda: api.kv_pages_alloc(pool, t, lens, i32(3)), lambda: api.kv_pages_fork(pool, t, lens, i32(1), i32(1)),
                 lambda: api.kv_pages_free(pool, t, lens, i32(2)), lambda: api.kv_pages_compact(pool, t, lens)):
        with pytest.raises(ValueError, match=DEVICE_ERR):
            call()
    with pytest.raises(ValueError, match="lens"):
        api.kv_pages_compact(pool, t, i32(2))
    with pytest.raises(TypeError, match="new_lens"):
        api.kv_pages_alloc(pool, t, lens, i32(3).long())
    with pytest.raises(ValueError, match="page_table"):
        api.kv_pages_free(pool, i32(24), lens, i32(1))
    moves = paged.page_moves([1], [2], 30, "cpu")
    with pytest.raises(ValueError, match="40 pages"):
        api.kv_pages_copy(cache(40), moves)
    with pytest.raises(ValueError, match="fork"):
        api.kv_tails_copy(torch.zeros(3, 2, 128, 32), moves)


@pytest.mark.parametrize("src,dst", [([0], [40]), ([-1], [0]), ([0, 1], [2]), ([0, 1], [2, 2]), ([0, 1], [1, 3])])
def test_page_moves_refuses_what_a_copy_in_any_order_cannot_do(src, dst):
    with pytest.raises(ValueError):
        paged.page_moves(src, dst, 40, "cpu")


# ---- the library ----
def test_struct_layouts(lib):
    assert lib.qk4v8_struct_size(4) == C.sizeof(_lib.Kv4Cache)
    assert lib.qk4v8_struct_size(5) == C.sizeof(_lib.Kv4Tokens)
    assert lib.qk4v8_struct_size(6) == C.sizeof(_lib.Kv4AttnParams)


def c_cache(**kw):
    a = dict(k_pages=FAKE, k_page_scales=FAKE, k_tensor_scale=FAKE, v_pages=FAKE, v_page_scales=FAKE,
             v_tensor_scale=FAKE, num_pages=40, kv_heads=2, head_dim=128)
    return _lib.Kv4Cache(**{**a, **kw})


BAD_CACHES = [(dict(k_pages=0), BAD), (dict(v_page_scales=0), BAD), (dict(v_tensor_scale=0), BAD), (dict(num_pages=0), BAD),
              (dict(kv_heads=0), BAD), (dict(kv_heads=65536), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED), (dict(v_pages=FAKE + 8), BAD),
              (dict(k_page_scales=FAKE + 4), BAD), (dict(k_tensor_scale=FAKE + 2), BAD)]


def test_token_call_validation(lib):
    def call(fn, cc=None, **kw):
        a = dict(cache=c_cache(**(cc or {})), k=FAKE, v=FAKE, k_stride=256, v_stride=512, dtype=1, total=9, cu=FAKE,
                 start=FAKE, page_table=FAKE, num_seqs=3, max_pages=8)
        return fn(C.byref(_lib.Kv4Tokens(**{**a, **kw})), None)
    for fn in (lib.kv4_append_paged, lib.kv4_read_paged):
        assert fn(None, None) == BAD
        assert call(fn, total=0) == 0                     # nothing to do, nothing launched
        assert call(fn, total=0, k=0, v=0) == 0
        for cc, want in BAD_CACHES:
            assert call(fn, cc) == want, cc
        for kw in (dict(k=0), dict(v=0), dict(cu=0), dict(start=0), dict(page_table=0), dict(k_stride=128), dict(v_stride=260),
                   dict(dtype=9), dict(total=-1), dict(num_seqs=0), dict(max_pages=0), dict(k=FAKE + 8), dict(v=FAKE + 2)):
            assert call(fn, **kw) == BAD, kw
        assert call(fn, dict(kv_heads=65535), k_stride=65535 * 128, v_stride=65535 * 128, total=2 ** 31 - 1) == UNSUPPORTED
    assert call(lib.kv4_append_paged, dtype=2) == BAD          # float32 can be read, not stored


def attn_params(cc=None, **kw):
    a = dict(cache=c_cache(**(cc or {})), q=FAKE, q_stride=8 * 128, dtype=1, total_q=6, cu_q=FAKE, context_lens=FAKE,
             page_table=FAKE, num_seqs=3, max_pages=8, q_heads=8, max_q=4, max_context=512, softmax_scale=0.1, out=FAKE, lse=0)
    return _lib.Kv4AttnParams(**{**a, **kw})


def test_attention_validation(lib):
    def call(cc=None, ws=FAKE, ws_bytes=1 << 40, **kw):
        return lib.attn_kv4_paged(C.byref(attn_params(cc, **kw)), ws, ws_bytes, None)
    assert lib.attn_kv4_paged(None, FAKE, 1 << 40, None) == BAD
    assert lib.attn_kv4_paged_workspace_size(None) == 0
    assert call(total_q=0) == 0 and call(total_q=0, q=0, out=0) == 0
    for cc, want in BAD_CACHES:
        if cc.get("kv_heads", 2) > 0:
            assert call(cc, q_heads=cc.get("kv_heads", 2) * 4, q_stride=cc.get("kv_heads", 2) * 512) == want, cc
    for kw in (dict(q=0), dict(out=0), dict(context_lens=0), dict(page_table=0), dict(dtype=2), dict(total_q=-1), dict(num_seqs=0),
               dict(max_pages=0), dict(q_heads=7), dict(q_heads=0), dict(max_q=0), dict(max_context=0), dict(max_context=513),
               dict(q_stride=1016), dict(q_stride=1028), dict(softmax_scale=0.0), dict(softmax_scale=-1.0),
               dict(softmax_scale=float("nan")), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(cu_q=0)):
        assert call(**kw) == BAD, kw
    assert call(q_heads=34, q_stride=34 * 128) == UNSUPPORTED                       # 17 heads a group
    assert call(num_seqs=1 << 20, max_pages=1 << 20, max_context=1 << 26) == UNSUPPORTED
    far = 2 ** 31 - 1                                     # more tiles than a CTA's range can count
    assert call(num_seqs=1, total_q=far, max_q=far, max_context=far, max_pages=1 << 26) == UNSUPPORTED
    for bad in (dict(ws=0), dict(ws=FAKE + 8), dict(ws_bytes=16)):
        assert call(**bad) == BAD, bad


def test_attention_workspace_grows_with_the_work_and_no_further(lib):
    def size(**kw):
        return lib.attn_kv4_paged_workspace_size(C.byref(attn_params(**kw)))
    step = dict(cu_q=0, max_q=1, total_q=64, num_seqs=64, max_pages=1 << 14)
    assert 0 < size(**step, max_context=64) <= size(**step, max_context=1 << 15) <= size(**step, max_context=1 << 20) < 1 << 23
    assert 0 < size(max_q=100, total_q=300) <= size(max_q=2000, total_q=6000) < 1 << 27
    assert size(q_stride=1028) == 0


def test_pool_validation(lib):
    n = lib.kv_pages_workspace_size(40, 3)
    assert n > 0 and lib.kv_pages_workspace_size(0, 3) == 0
    base = (FAKE, 40, FAKE, 3, 8, FAKE)

    def bases():
        for at, v in ((0, 0), (1, 0), (2, 0), (3, 0), (4, 0), (5, 0), (0, FAKE + 2), (1, -1)):
            yield base[:at] + (v,) + base[at + 1:]
    for b in bases():
        assert lib.kv_pages_alloc(*b, FAKE, FAKE, n, None) == BAD, b
        assert lib.kv_pages_fork(*b, FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == BAD, b
        assert lib.kv_pages_free(*b, FAKE, 1, None) == BAD, b
        assert lib.kv_pages_compact(*b, FAKE, FAKE, FAKE, FAKE, n, None) == BAD, b
    assert lib.kv_pages_alloc(*base, 0, FAKE, n, None) == BAD
    assert lib.kv_pages_alloc(*base, FAKE, FAKE, n - 1, None) == BAD
    assert lib.kv_pages_fork(*base, FAKE, FAKE, -1, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == BAD
    assert lib.kv_pages_fork(*base, 0, 0, 0, 0, 0, 0, 0, FAKE, n, None) == 0
    assert lib.kv_pages_fork(*base, FAKE, FAKE, 1, FAKE, FAKE, 0, FAKE, FAKE, n, None) == BAD
    assert lib.kv_pages_free(*base, 0, 0, None) == 0 and lib.kv_pages_free(*base, 0, 1, None) == BAD
    assert lib.kv_pages_compact(*base, FAKE, 0, FAKE, FAKE, n, None) == BAD
    arr, size = (C.c_void_p * 2)(FAKE, FAKE), (C.c_int64 * 2)(4096, 512)
    assert lib.kv_pages_copy(arr, size, 2, 40, FAKE, FAKE, 0, None, None) == 0
    assert lib.kv_pages_copy(arr, size, 0, 40, FAKE, FAKE, 1, None, None) == BAD
    assert lib.kv_pages_copy(arr, size, 9, 40, FAKE, FAKE, 1, None, None) == BAD
    assert lib.kv_pages_copy(arr, (C.c_int64 * 2)(4096, 24), 2, 40, FAKE, FAKE, 1, None, None) == BAD
    assert lib.kv_pages_copy((C.c_void_p * 2)(FAKE, FAKE + 8), size, 2, 40, FAKE, FAKE, 1, None, None) == BAD
    assert lib.kv_pages_copy(arr, size, 2, 40, 0, FAKE, 1, None, None) == BAD


# ---- the oracle ----
def test_oracle_cache_keeps_each_token_apart():
    rng = np.random.default_rng(0)
    c = OK.Cache(4, 2, 128, 2.0 ** -5, 2.0 ** -7)
    k, v = rng.standard_normal((2, 130, 2, 128)).astype(np.float32)
    row = [3, 0, 2]
    for a, b in ((0, 1), (1, 64), (64, 67), (67, 130)):   # whatever the cuts, the same pages
        c.append(k[a:b], v[a:b], a, row)
    whole = OK.Cache(4, 2, 128, 2.0 ** -5, 2.0 ** -7)
    whole.append(k, v, 0, row)
    for x, y in ((c.kp, whole.kp), (c.ks, whole.ks), (c.vp, whole.vp), (c.vs, whole.vs)):
        assert (x == y).all()
    rk, rv = c.read(130, row)
    # a value's error: half the largest step of its block (2 of 6), with the block scale's own half step
    for x, r, ts in ((k, rk, 2.0 ** -5), (v, rv, 2.0 ** -7)):
        amax = np.abs(x.reshape(130, 2, 8, 16)).max(-1, keepdims=True)
        assert (np.abs(x - r).reshape(130, 2, 8, 16) <= amax * (1 / 6 + 2.0 ** -4) + ts * 2.0 ** -9).all()
    # one token by hand: page 0 (position 65), head 1, channels 16 .. 31
    byte = c.vp[0, 1, 0, 16:32] >> 4
    assert (rv[65, 1, 16:32] == e2m1_decode(byte) * e4m3_decode(c.vs[0, 1, 1, 1]) * 2.0 ** -7).all()
    a, b = c.read(3, row, 64)
    assert (a == rk[64:67]).all() and (b == rv[64:67]).all()


def test_oracle_attention_is_a_causal_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, lse = OK.attention(q, k, v, 0.5)
    for i in range(2):
        for h in range(4):
            s = [0.5 * float(q[i, h] @ k[j, h // 2]) for j in range(4 + i)]
            z = sum(math.exp(x) for x in s)
            want = sum(math.exp(x) / z * v[j, h // 2] for j, x in enumerate(s))
            assert np.allclose(out[i, h], want, atol=1e-12) and abs(lse[i, h] - math.log(z)) < 1e-12
