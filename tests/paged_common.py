"""Shared helpers of the paged-cache tests: pools with known contents, calls
through the binding, and the tolerances of the attention."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged_oracle as P
from quantized_kv_cache_quantize_gb300 import kvq


def random_pool(seed, layers, n_pages, heads, page, d, e_lo=-9, e_hi=-3, nan_pages=False):
    """Codes of any finite value (or, for pages nothing may read, NaN) and a
    scale of its own per page and head; CPU tensors."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(2):
        x = rng.standard_normal((layers, n_pages, heads, page, d)) * 100
        c = P.e4m3_code(P.e4m3_round(x))
        if nan_pages:
            c[:] = 0x7F
        out.append(torch.from_numpy(c))
    exps = [rng.integers(e_lo, e_hi + 1, (layers, n_pages, heads)) for _ in range(2)]
    return out, exps


def scale_tensor(exps) -> torch.Tensor:
    return torch.from_numpy(2.0 ** np.asarray(exps, np.float64)).to(torch.bfloat16)


def cache_of(codes, exps, device="cuda") -> kvq.PagedCache:
    return kvq.PagedCache(*[c.to(device).view(torch.float8_e4m3fn) for c in codes],
                          *[scale_tensor(e).to(device) for e in exps])


def codes_of(t: torch.Tensor) -> np.ndarray:
    return t.view(torch.uint8).cpu().numpy()


def exps_of(t: torch.Tensor) -> np.ndarray:
    s = t.float().cpu().numpy().astype(np.float64)
    e = np.rint(np.log2(s)).astype(np.int64)
    assert np.array_equal(2.0 ** e, s)
    return e


def make_table(rng, lens, page, n_pages, width=None, fill=-1):
    """Distinct pages in no order; `fill` in the entries past each length."""
    need = [-(-int(n) // page) for n in lens]
    width = max(need + [1]) if width is None else width
    ids = rng.permutation(n_pages)
    assert sum(need) <= n_pages
    t = np.full((len(lens), width), fill, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = ids[at:at + k]
        at += k
    return t


def offsets_of(counts) -> torch.Tensor:
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def dev(t, dtype=torch.int32):
    return torch.as_tensor(np.asarray(t)).to(dtype).cuda()


def tolerances(out, lse, bound, serr, qerr, d, n_keys):
    """How far out and lse may be from the 64-bit answer, element by element.
    The codes and scales are exact operands; what rounds is
    - a query element far below its row's largest: as two E4M3 parts with the
      largest magnitude at 2^7 or above, an element is off by half a step of
      the subnormals at most, 2^-10, so by 2^-17 of the largest (as FP16 with
      the largest at 2^14 or above: 2^-39);
    - a score: d products summed in fp32 (d + 1 roundings, at 2^-23 each
      because the tensor core may truncate) and the multiplications by the
      scales and log2 e (3 more), all relative to sum |q k|, plus its 2^x
      (2^-21 relative, the special-function unit's bound doubled);
      a shift ds of a score moves p by a factor e^ds, and its sum likewise:
      2 ds relative;
    - p as a 16-bit operand: 2^-11 (FP16, half a step); FP16 subnormals add
      2^-25 a key, n_keys of them at most, where the largest weight stands at
      2^9 or above: 2^-34 of it;
    - sums of n_keys terms in fp32: n_keys 2^-23, relative to sum p |v|;
    - the BF16 output: 2^-8 (half a step) of the value.
    lse: the score's shift, the fp32 sum, and its own representation."""
    ds = (d + 4) * 2.0 ** -23 * serr + 2.0 ** -17 * qerr + 2.0 ** -21
    rel = 2 * ds + 2.0 ** -11 + n_keys * 2.0 ** -23 + n_keys * 2.0 ** -34
    tol_o = (2.0 ** -8) * (np.abs(out) + rel[..., None] * bound) + rel[..., None] * bound
    tol_l = ds + n_keys * 2.0 ** -23 + 2.0 ** -21 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22
    return tol_o, tol_l


def check_attention(got, ref, d, n_keys, what=""):
    out, lse, bound, serr, qerr = ref
    o = got[0].float().cpu().numpy().astype(np.float64)
    z = got[1].cpu().numpy().astype(np.float64)
    tol_o, tol_l = tolerances(out, lse, bound, serr, qerr, d, n_keys)
    assert np.isfinite(o).all(), what
    empty = ~np.isfinite(lse)
    assert np.array_equal(z == -np.inf, empty), what
    assert (o[empty] == 0).all(), what
    over = np.abs(o - out) > tol_o
    assert not over.any(), (what, "out", int(over.sum()), float((np.abs(o - out) / np.maximum(tol_o, 1e-300)).max()))
    far = np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse)) > tol_l
    assert not far.any(), (what, "lse", int(far.sum()), float(np.nanmax(np.abs(z - lse))))
