"""Set up paged KV caches (NVFP4-K / MXFP8-V, and the 4-bit one) and their page pool; fill a
paged NVFP4-K / MXFP8-V KV cache from dense per-sequence K/V.

Quantization runs in the library's kernels (quantize_nvfp4 with the cache's fixed tensor
scale, quantize_mxfp8_v); torch only moves the resulting bytes into 64-token pages at the
physical ids of the page table. This is cache set-up, outside the decode step.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from .api import PagedKV, PagedKV4, PageMoves, quantize_mxfp8_v, quantize_nvfp4

PAGE = 64


def empty_cache(num_pages: int, kv_heads: int, head_dim: int, k_tensor_scale: float,
                device) -> PagedKV:
    d = head_dim
    return PagedKV(
        k_pages=torch.zeros(num_pages, kv_heads, PAGE, d // 2, dtype=torch.uint8, device=device),
        k_scales=torch.zeros(num_pages, kv_heads, PAGE, d // 16, dtype=torch.uint8, device=device),
        k_tensor_scale=torch.tensor([k_tensor_scale], dtype=torch.float32, device=device),
        v_pages=torch.zeros(num_pages, kv_heads, d, PAGE, dtype=torch.uint8, device=device),
        v_scales=torch.full((num_pages, kv_heads, d, 2), 127, dtype=torch.uint8, device=device),
    )


def empty_cache4(num_pages: int, kv_heads: int, head_dim: int, k_tensor_scale: float,
                 v_tensor_scale: float, device) -> PagedKV4:
    """A zeroed 4-bit cache. A tensor scale of s covers values up to 2688 s."""
    d, u8 = head_dim, dict(dtype=torch.uint8, device=device)
    return PagedKV4(
        k_pages=torch.zeros(num_pages, kv_heads, PAGE, d // 2, **u8),
        k_scales=torch.zeros(num_pages, kv_heads, PAGE, d // 16, **u8),
        k_tensor_scale=torch.tensor([k_tensor_scale], dtype=torch.float32, device=device),
        v_pages=torch.zeros(num_pages, kv_heads, PAGE // 2, d, **u8),
        v_scales=torch.zeros(num_pages, kv_heads, d // 16, PAGE, **u8),
        v_tensor_scale=torch.tensor([v_tensor_scale], dtype=torch.float32, device=device),
    )


@dataclass
class PagePool:
    """Which pages of a cache are in use: refs [num_pages] int32, the number of sequences that
    hold each page (0 = free). Used by api.kv_pages_alloc, _fork, _free and _compact."""
    refs: torch.Tensor


def empty_pool(num_pages: int, device) -> PagePool:
    return PagePool(torch.zeros(num_pages, dtype=torch.int32, device=device))


def page_moves(src, dst, num_pages: int, device) -> PageMoves:
    """Page copies of the caller's own choice (lists of page numbers) for api.kv_pages_copy.
    Refuses numbers out of range, a destination given twice and one that is also a source."""
    src, dst = [int(p) for p in src], [int(p) for p in dst]
    if len(src) != len(dst):
        raise ValueError("src and dst must have the same length")
    if any(not 0 <= p < num_pages for p in src + dst):
        raise ValueError(f"page numbers must be in 0..{num_pages - 1}")
    if len(set(dst)) != len(dst) or set(dst) & set(src):
        raise ValueError("a destination page is given twice or is also a source")
    t = torch.tensor([src, dst], dtype=torch.int32, device=device)
    return PageMoves(t[0], t[1], num_pages)


def empty_tail(num_seqs: int, kv_heads: int, head_dim: int, dtype, device) -> torch.Tensor:
    """The per-sequence incomplete-V-group state that kv_append_paged reads and updates."""
    return torch.zeros(num_seqs, kv_heads, head_dim, 32, dtype=dtype, device=device)


def write_sequence(cache: PagedKV, k: torch.Tensor, v: torch.Tensor, pages: torch.Tensor) -> None:
    """Quantize one sequence's K, V ([len, Hkv, D] on the cache's device) into the physical
    pages ``pages`` (int tensor of ceil(len/64) ids)."""
    n, hkv, d = k.shape
    n_pages = (n + PAGE - 1) // PAGE
    npad = n_pages * PAGE
    kh = torch.zeros(hkv, npad, d, dtype=k.dtype, device=k.device)
    kh[:, :n] = k.transpose(0, 1)
    k4 = quantize_nvfp4(kh, tensor_scale=float(cache.k_tensor_scale.item()))
    pages = pages.to(device=k.device, dtype=torch.long)
    cache.k_pages[pages] = k4.codes.view(hkv, n_pages, PAGE, d // 2).transpose(0, 1)
    cache.k_scales[pages] = k4.scales.view(hkv, n_pages, PAGE, d // 16).transpose(0, 1)
    v8 = quantize_mxfp8_v(v.transpose(0, 1).contiguous())          # codes [Hkv, D, n_pad128]
    vc = v8.codes[:, :, :npad].reshape(hkv, d, n_pages, PAGE).permute(2, 0, 1, 3)
    vs = v8.scales[:, :, :npad // 32].reshape(hkv, d, n_pages, 2).permute(2, 0, 1, 3)
    cache.v_pages[pages] = vc
    cache.v_scales[pages] = vs
