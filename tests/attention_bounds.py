"""How far attention over the cache may be off, kernel by kernel, and a case run
against it.

With A = sum_j p_j |v_j|, E the largest scale * sum_d |q_d k_jd| and L the
positions, of a row; a rounding to f16 is off by 2^-11 of the value at most, one
to f32 by 2^-24:
  * score: what q or the key loses on its way to the matrix cores (`KEYS`), the D
    products and their scales in f32, (D + 8) 2^-24, both times E; a cap keeps
    relative accuracy, |c(x)| <= |x|: 2^-20 E with one; the exponent's argument
    from score and running maximum 2^-22 (E + 4), exp2 2^-22;
  * probability: relative error twice the score's, as their sum has it too, and
    what its own rounding costs (`PROBABILITIES`);
  * value: rounded to f16 by the kernel for many rows (`VALUES`), unless it is a
    number that f16 holds;
  * where f16 ends: f16 is off by 2^-25 at most below 2^-14.  Rows kernel: P d is
    kept so that the largest d met lies in [2^13, 2^14), and a block of largest d
    has a code of 127 (Q8_0) or 8 (Q4_0) with no other code above: 2^-38 of the
    largest value.  Kernel for many rows: P is 2^6 or more at the row's largest,
    so 2^-31; value scales are kept so that the largest lies in [2^7, 2^8): 2^-32.
    Each of L positions, over a sum of 1 or more;
  * sums over L positions in f32: (L / 16 + 16) 2^-24 A;
  * one rounding to the output's type.
lse: the scores' error (probabilities are summed before they are rounded), the
sum's (L / 16 + 16) 2^-24, and what log2 and two f32 steps cost, 2^-22 (|lse| +
E + 4).
"""
import numpy as np
import torch

import block_quantized_matmul_gguf_amd as qmm
import cache_ref as ref
from test_gpu_attention import TYPES, check, gpu, largest, starts_of

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# f32: two f16 parts of the row's power of two, 2^-21 of its largest value, which is 2^-19 of E (see
# test_gpu_attention.py); f16 and bf16 enter as they are, but for bits 2^-31 below the largest.  Keys are exact codes
# in the rows kernel; code * d in two parts or one in the other, with a part that f16 does not hold, 2^-32 of the
# largest: 2^-26 E covers both where neither the row nor the keys span more than 2^5 sums' worth.
KEYS = {("rows", F32): 2.0**-19, ("rows", F16): 2.0**-26, ("rows", BF16): 2.0**-26, ("many", F16): 2.0**-26, ("many", BF16): 2.0**-11}
PROBABILITIES = {("rows", F32): 2.0**-21, ("rows", F16): 2.0**-11, ("rows", BF16): 2.0**-11, ("many", F16): 2.0**-21,
                 ("many", BF16): 2.0**-11}
VALUES = {"rows": 0.0, "many": 2.0**-11}
ENDS = {"rows": 2.0**-37, "many": 2.0**-30}


def bounds(kernel, dt, dim, length, big, top, most, lse, capped=False, exact_values=False):
    """(of out [n, Hq, D] before its rounding, of lse [n, Hq])"""
    s = top * (KEYS[kernel, dt] + (dim + 8) * 2.0**-24 + capped * 2.0**-20) + 2.0**-22 * (top + 4) + 2.0**-22
    sums = (length / 16 + 16) * 2.0**-24
    values = 0.0 if exact_values else VALUES[kernel]
    out = big * (np.expm1(2 * s)[..., None] + PROBABILITIES[kernel, dt] + values + sums) + length * ENDS[kernel] * most
    with np.errstate(invalid="ignore"):
        of_lse = np.where(np.isfinite(lse), s + sums + 2.0**-22 * (np.abs(lse) + top + 4), 0.0)
    return out, of_lse


def run_close(kernel, c, dtype, per, new, seed=0, q_scale=1.0, scale=None, causal=True, window=0, softcap=0.0, max_length=0,
              exact_values=False):
    """One call over the cache c (`cache_ref.Cache`) checked against the bounds; (out, lse)."""
    dt, dim, heads, lengths = TYPES[dtype], c.dim, c.heads * per, c.lengths
    st = starts_of(new)
    q = np.random.default_rng(seed).standard_normal((int(st[-1]), heads, dim)) * q_scale
    q = torch.from_numpy(q.astype(np.float32)).to(dt)
    lse = torch.empty(q.shape[:2], dtype=F32, device="cuda")
    out = qmm.cache_attention(c.fmt_k, c.fmt_v, gpu(c.k_cache), gpu(c.v_cache), q.cuda(), gpu(c.table), gpu(st), gpu(lengths),
                              scale=scale, causal=causal, window=window, softcap=softcap, max_length=max_length, lse=lse)
    for s, n in enumerate(lengths):
        if not new[s]:
            continue
        rows = slice(st[s], st[s + 1])
        o, l, big, top = ref.attention(q[rows].double().numpy(), c.kq[s], c.vq[s], np.arange(n - new[s], n),
                                       dim ** -0.5 if scale is None else scale, causal, window, softcap)
        tol, of_lse = bounds(kernel, dt, dim, min(int(n), window or int(n)), big, top, largest(c.vq[s]), l, softcap > 0, exact_values)
        check(out[rows], o, tol, f"out of sequence {s}")
        check(lse[rows], l, of_lse, f"lse of sequence {s}")
    return out, lse
