"""Plain fp64 reference of the windowed attention and of the read-back, on a host copy of
the packed pages: codes and levels from the oracle, rotation as an explicit matrix,
attention as a softmax over the visible tokens.  Also the error bounds that the tests use.
"""
from __future__ import annotations

import numpy as np

PAGE = 64
EPS_HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def rotation_matrices(oracle, params64, d, rot=0):
    """R [H][d][d] with rotated = R x."""
    eye = np.eye(d)
    return np.stack([np.stack([oracle.rotate(p, eye[i], rot) for i in range(d)], 1)
                     for p in params64])


def _norms(blocks, off):
    return blocks[..., off:off + 2 * PAGE].copy().view(np.float16).astype(np.float64)


def dequantize_pages(oracle, params64, blocks, d, bits=3, rot=0):
    """K, V [P][64][H][d] and their rotated forms kt, vt of every page (norms that are not
    finite give non-finite vectors)."""
    P, H = blocks.shape[:2]
    cb = bits * d // 8
    lev = np.asarray(oracle.levels(bits))
    R = rotation_matrices(oracle, params64, d, rot)
    kc = oracle.unpack_codes_batch(blocks[..., :PAGE * cb].reshape(P, H, PAGE, cb), d, bits=bits)
    v_at = PAGE * (cb + 2)
    reg = np.ascontiguousarray(blocks[..., v_at:v_at + PAGE * cb])
    vc = oracle.unpack_codes_batch(oracle.v_region_records(reg, d, bits=bits), d, bits=bits)
    with np.errstate(invalid="ignore"):
        kt = lev[kc] * (_norms(blocks, PAGE * cb) / np.sqrt(d))[..., None]
        vt = lev[vc] * (_norms(blocks, v_at + PAGE * cb) / np.sqrt(d))[..., None]
        K = np.einsum("phse,hed->pshd", kt, R)
        V = np.einsum("phse,hed->pshd", vt, R)
    return K, V, kt.transpose(0, 2, 1, 3), vt.transpose(0, 2, 1, 3), R


def visible(p, window, sinks):
    """Positions that a query at position p sees, ascending."""
    if p < 0:
        return np.zeros(0, np.int64)
    lo = max(0, p + 1 - window)
    return np.concatenate([np.arange(min(sinks, lo, p + 1)), np.arange(lo, p + 1)]).astype(np.int64)


def window_attention(pages, page_table, lens, Q, scale, window, sinks, bits=3, out="f32"):
    """Q [n_seqs][n_q][hq][d] -> (reference, row error bound), both per row.

    The bound, as an L2 norm per row (B = sum p |v|, T visible tokens, every term an upper
    bound of what the kernels round):
      2^-11 B       the weights p |v| / sigma as binary16 operands (half a step)
      T 2^-25 2.2 v weights below binary16's smallest normal: half a subnormal step each,
                    times the largest |V| and the largest level 2.152 (2.7326 at 4 bits, and
                    1.52 at 2: taken as 2.8)
      eL B          the value levels as binary16: 2e-5 (3 bits), 0 (2 bits), 6e-5 (4 bits)
      2 dS B        an error dS of every score changes a softmax weight by at most a factor
                    exp(2 dS); dS = eS max_t scale sum |q~ k~| with eS = eL for the levels of
                    the f16 scores, plus 2^-18 for the query's parts, the products' sums and
                    the exponential
      (T/16+8) 2^-23 B  fp32 sums over the tokens, a block of 16 at a time, and the merges
      half a step of the output type, relative to each element.
    """
    K, V, kt, vt, R = pages
    n_seqs, n_q, hq, d = Q.shape
    H = K.shape[2]
    G = hq // H
    eL = {2: 0.0, 3: 2e-5, 4: 6e-5}[bits]
    ref, tol = np.zeros(Q.shape), np.zeros(Q.shape[:-1])
    for s in range(n_seqs):
        for i in range(n_q):
            t = visible(int(lens[s]) - n_q + i, window, sinks)
            if not len(t):
                continue
            ph = page_table[s, t // PAGE]
            for h in range(H):
                k, v = K[ph, t % PAGE, h], V[ph, t % PAGE, h]
                q = Q[s, i, h * G:(h + 1) * G]
                x = q @ k.T * scale
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ v
                vn = np.linalg.norm(v, axis=-1)
                B = p @ vn
                dS = (eL + 2.0 ** -18) * scale * (np.abs(q @ R[h].T) @ np.abs(kt[ph, t % PAGE, h]).T).max(-1)
                T = len(t)
                ref[s, i, h * G:(h + 1) * G] = o
                tol[s, i, h * G:(h + 1) * G] = (
                    (2.0 ** -11 + eL + 2 * dS + (T / 16 + 8) * 2.0 ** -23) * B
                    + T * 2.0 ** -25 * 2.8 * vn.max() + EPS_HALF[out] * np.linalg.norm(o, axis=-1))
    return ref, tol
