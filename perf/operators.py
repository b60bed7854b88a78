"""What is measured of the packed cache's windowed attention and of its read-back.

Three operators on the paged cache of packed codes (include/isoq.h gives the layout):

  decode   one query token per sequence attends the last `window` tokens and the first
           `sinks` tokens of its context; pages in between have been recycled
  chunk    the same for a chunk of query tokens per sequence, each with its own window
           (chunked prefill, verification of drafted tokens)
  read     K and V of listed tokens read back from the codes, with the rotary embedding
           of K taken off where `rope` is set

``run`` computes them in elementary torch operations in 32 bits (``own`` false) or through
the framework's entry points (``own`` true) from the same state.  ``exact`` is the
definition in 64 bits, from the bit positions of the codes and explicit rotation matrices.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
PARAM_SEED = 0
ROPE_BASE = 10000.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# Lloyd-Max quantisers for N(0,1) (J. Max, 1960): the non-negative levels by bits per code
MAGS = {2: [0.4528, 1.5104],
        3: [0.2451, 0.7560, 1.3440, 2.1520],
        4: [0.1284, 0.3881, 0.6568, 0.9424, 1.2562, 1.6180, 2.0690, 2.7326]}


# ---- cases -------------------------------------------------------------------------------
def _attention(name, op, n_seqs, lens, heads, kv_heads, window, sinks, n_q=1, d=128, bits=3,
               q="bf16", out="bf16"):
    return {"name": name, "op": op, "n_seqs": n_seqs, "len_lo": lens[0], "len_hi": lens[1],
            "heads": heads, "kv_heads": kv_heads, "window": window, "sinks": sinks, "n_q": n_q,
            "d": d, "bits": bits, "q": q, "out": out}


def _read(name, n_seqs, length, tokens, kv_heads, d=128, bits=3, out="bf16", rope=False,
          shuffled=False):
    return {"name": name, "op": "read", "n_seqs": n_seqs, "len": length, "tokens": tokens,
            "kv_heads": kv_heads, "d": d, "bits": bits, "out": out, "rope": rope,
            "shuffled": shuffled}


def listed():
    return [
        # one user's chat past 32k tokens, a short window: the smallest decode step
        _attention("decode_1seq_w1024", "decode", 1, (32768, 32768), 32, 4, 1024, 4),
        # eight long conversations with their old pages recycled
        _attention("decode_8seq_131k_w4096", "decode", 8, (131072, 131072), 64, 8, 4096, 4),
        # a full serving batch of ragged lengths, one page of sinks: the largest decode step
        _attention("decode_64seq_ragged_w8192", "decode", 64, (4096, 65536), 32, 8, 8192, 64,
                   q="f16", out="f16"),
        # the wide head dimension, a window and sinks that end inside pages
        _attention("decode_4seq_d256_w2000", "decode", 4, (32000, 32768), 16, 8, 2000, 5, d=256),
        # 4-bit codes, fp32 queries, odd heads, sequences from empty to longer than the window
        _attention("decode_9seq_4bit_w777", "decode", 9, (0, 3000), 15, 3, 777, 3, bits=4,
                   q="f32"),
        # five drafted tokens per sequence to verify
        _attention("chunk_16seq_5tok_w4096", "chunk", 16, (8192, 65536), 32, 8, 4096, 4, n_q=5),
        # a 16-token chunk per long conversation
        _attention("chunk_8seq_16tok_w4096", "chunk", 8, (131072, 131072), 64, 8, 4096, 4,
                   n_q=16),
        # chunked prefill of a long prompt: the most arithmetic
        _attention("chunk_1seq_2048tok_w4096", "chunk", 1, (32768, 32768), 64, 8, 4096, 4,
                   n_q=2048),
        # one page handed to another path
        _read("read_1page", 1, 4096, 64, 8),
        # a 32k prefix read back for a full-precision consumer: the most bytes
        _read("read_prefix_32k", 1, 32768, 32768, 8),
        # keys without their rotary embedding, to be placed at other positions
        _read("read_rope_d256_5001", 2, 4096, 5001, 8, d=256, out="f16", rope=True),
        # tokens picked across sequences, in any order, to fp32
        _read("read_picked_4bit_f32", 5, 4001, 10007, 3, bits=4, out="f32", shuffled=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "chunk", "read"])
    d = rng.choice([128, 128, 128, 256])
    bits = rng.choice([3, 3, 3, 2, 4]) if d == 128 else 3
    if op == "read":
        n_seqs = _log_int(rng, 1, 16)
        tokens = _log_int(rng, 1, 16384)
        length = -(-tokens // n_seqs) + rng.randrange(0, 200)
        return _read("", n_seqs, length, tokens, rng.choice([1, 2, 3, 4, 8]), d=d, bits=bits,
                     out=rng.choice(["bf16", "f16", "f32"]), rope=rng.random() < 0.4,
                     shuffled=rng.random() < 0.4)
    heads, kv_heads = rng.choice([(8, 2), (32, 4), (32, 8), (64, 8), (15, 3), (7, 7), (16, 1)])
    if d == 256:
        heads, kv_heads = rng.choice([(16, 8), (8, 2), (6, 3)])
    window, sinks = _log_int(rng, 16, 8192), rng.choice([0, 1, 4, 5, 64, 100])
    hi = _log_int(rng, 32, 131072)
    lo = rng.choice([0, hi // 2, hi])
    q, out = rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "f16"])
    if op == "decode":
        return _attention("", op, _log_int(rng, 1, 64), (lo, hi), heads, kv_heads, window, sinks,
                          d=d, bits=bits, q=q, out=out)
    n_q = _log_int(rng, 2, 1024) if d == 128 else _log_int(rng, 2, 64)
    # no more (query row, key) pairs than the listed prefill has
    room = (64 * 2048 * 4096) // (heads * n_q * (window + sinks + n_q))
    n_seqs = _log_int(rng, 1, max(1, min(32, room)))
    return _attention("", op, n_seqs, (lo, hi), heads, kv_heads, window, sinks, n_q=n_q, d=d,
                      bits=bits, q=q, out=out)


# ---- what a user's program has in hand ---------------------------------------------------
def _splitmix64(seed, n):
    """The first n outputs of SplitMix64 (Steele, Lea & Flood, 2014)."""
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + np.arange(1, n + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def _quaternions(d, kv_heads):
    """The rotation parameters of seed PARAM_SEED as binary32: [kv_heads][d/4][p, q][4]."""
    u = (_splitmix64(PARAM_SEED, kv_heads * d * 4) >> np.uint64(11)).astype(np.float64)
    u = u.reshape(-1, 2)
    g = np.sqrt(-2.0 * np.log((u[:, 0] + 1.0) * 2.0 ** -53)) * np.cos(2 * np.pi * u[:, 1] * 2.0 ** -53)
    g = g.reshape(kv_heads, d // 4, 2, 4)
    return (g / np.sqrt((g * g).sum(-1, keepdims=True))).astype(np.float32)


def _hamilton(a, b):
    aw, ax, ay, az = np.moveaxis(a, -1, 0)
    bw, bx, by, bz = np.moveaxis(b, -1, 0)
    return np.stack([aw * bw - ax * bx - ay * by - az * bz, aw * bx + ax * bw + ay * bz - az * by,
                     aw * by - ax * bz + ay * bw + az * bx, aw * bz + ax * by - ay * bx + az * bw], -1)


def _rotation(d, kv_heads):
    """R [kv_heads][d][d] in 64 bits: the rotated vector is R x (orthonormal WHT, then the
    4x4 blocks p y conj(q))."""
    pq = _quaternions(d, kv_heads).astype(np.float64)
    p, qc = pq[:, :, 0], pq[:, :, 1] * np.array([1.0, -1.0, -1.0, -1.0])
    had = np.ones((1, 1))
    while had.shape[0] < d:
        had = np.block([[had, had], [had, -had]])
    R = np.zeros((kv_heads, d, d))
    for j in range(4):
        unit = np.broadcast_to(np.eye(4)[j], p.shape)
        col = _hamilton(_hamilton(p, unit), qc)          # [kv_heads][d/4][4]
        for i in range(4):
            for b in range(d // 4):
                R[:, 4 * b + i, :] += col[:, b, i, None] * had[4 * b + j] / math.sqrt(d)
    return R


_rotations = {}


def _rotation_of(d, kv_heads):
    if (d, kv_heads) not in _rotations:
        _rotations[d, kv_heads] = _rotation(d, kv_heads)
    return _rotations[d, kv_heads]


def _levels(bits):
    return [-m for m in reversed(MAGS[bits])] + MAGS[bits]


def _slot2():
    """2-bit layout: the slot of dims 0..15 of a word."""
    return [(e % 8) // 2 + 4 * (e % 2) + 8 * (e // 8) for e in range(16)]


def _pack_rows(codes, bits):
    """Codes [..., d] (int64) of one record per slot -> int32 words [..., bits * d / 32]."""
    shape, dev = codes.shape[:-1], codes.device
    if bits == 3:
        c = codes.reshape(*shape, -1, 4, 8)
        spare = torch.stack([(c[..., 3, :] >> (2 - b)) & 1 for b in range(3)], -2)
        words = ((c[..., :3, :] | (spare << 3)) << (4 * torch.arange(8, device=dev))).sum(-1)
    elif bits == 4:
        c = codes.reshape(*shape, -1, 8)
        words = (torch.where(c >= 8, c - 8, 15 - c) << (4 * torch.arange(8, device=dev))).sum(-1)
    else:
        c = codes.reshape(*shape, -1, 16)
        words = (c << (2 * torch.tensor(_slot2(), device=dev))).sum(-1)
    return words.to(torch.int32).reshape(*shape, -1)


def _pack_v3(codes):
    """3-bit V codes of whole pages [P, H, 64, d] -> words [P, H, 6 d]: the V tile layout."""
    P, H, _, d = codes.shape
    c = codes.reshape(P, H, 4, 2, 4, 2, d // 16, 2, 4, 2)    # block, j1, t, j0, u1, u0, b, e
    c = c.permute(0, 1, 2, 6, 4, 7, 8, 9, 3, 5).reshape(P, H, 4, d // 16, 4, 2, 4, 8)
    spare = torch.stack([(c[..., 3, :] >> (2 - b)) & 1 for b in range(3)], -2)
    shift = 4 * torch.arange(8, device=codes.device)         # nibble e * 4 + 2 j1 + j0
    words = ((c[..., :3, :] | (spare << 3)) << shift).sum(-1)
    return words.to(torch.int32).reshape(P, H, 6 * d)


def _quantize(x, R, bits):
    """Vectors [P, 64, H, d] -> codes [P, H, 64, d] (int64), norms [P, H, 64] (f16)."""
    d = x.shape[-1]
    z = torch.einsum("pshd,hed->phse", x, R).contiguous()
    n = torch.linalg.vector_norm(x, dim=-1).transpose(1, 2).contiguous()
    lev = torch.tensor(_levels(bits), device=x.device)
    codes = torch.bucketize(z * (math.sqrt(d) / n[..., None]), (lev[1:] + lev[:-1]) / 2, right=True)
    return codes, n.to(torch.float16)


def _fill_pages(g, n_pages, kv_heads, d, bits):
    """Packed pages of tokens with per-channel scales log-uniform in [0.1, 10]."""
    dev = g.device
    R = torch.tensor(_rotation_of(d, kv_heads), dtype=torch.float32, device=dev)
    scales = [torch.exp(torch.empty((kv_heads, d), device=dev).uniform_(
        math.log(0.1), math.log(10.0), generator=g)) for _ in range(2)]
    parts = []
    for p0 in range(0, n_pages, 1024):
        P = min(1024, n_pages - p0)
        fields = []
        for side in range(2):
            x = torch.randn((P, PAGE, kv_heads, d), generator=g, device=dev) * scales[side]
            codes, norms = _quantize(x.to(torch.bfloat16).float(), R, bits)
            words = _pack_v3(codes) if side and bits == 3 else _pack_rows(codes, bits)
            fields += [words.reshape(P, kv_heads, -1).view(torch.uint8), norms.view(torch.uint8)]
        parts.append(torch.cat(fields, -1))
    return torch.cat(parts)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1_000_003 * seed + 17)
    cpu = torch.Generator()
    cpu.manual_seed(1_000_033 * seed + 29)
    c, d, H, bits = case, case["d"], case["kv_heads"], case["bits"]
    n_seqs = c["n_seqs"]
    if c["op"] == "read":
        lens = torch.full((n_seqs,), c["len"])
        first_kept, sink_pages = torch.zeros_like(lens), torch.zeros_like(lens)
    else:
        lens = torch.randint(c["len_lo"], c["len_hi"] + 1, (n_seqs,), generator=cpu)
        first_kept = (lens - c["n_q"] + 1 - c["window"]).clamp(min=0) // PAGE
        sink_pages = (lens.clamp(max=c["sinks"]) + PAGE - 1) // PAGE
    # the pages that the attention can still reach are kept; the others have been recycled
    max_pages = max(1, -(-int(lens.max()) // PAGE))
    page = torch.arange(max_pages)
    kept = (page < (lens[:, None] + PAGE - 1) // PAGE) & (
        (page >= first_kept[:, None]) | (page < sink_pages[:, None]))
    n_pages = max(1, int(kept.sum()))
    page_table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32)
    page_table[kept] = torch.randperm(n_pages, generator=cpu)[:int(kept.sum())].to(torch.int32)
    s = {"case": dict(case), "page_table": page_table.to(dev),
         "blocks": _fill_pages(g, n_pages, H, d, bits),
         "R": torch.tensor(_rotation_of(d, H), dtype=torch.float32, device=dev),
         "status": torch.zeros((1,), dtype=torch.int32, device=dev)}
    if c["op"] == "read":
        every = n_seqs * c["len"]
        at = torch.randperm(every, generator=cpu)[:c["tokens"]] if c["shuffled"] else torch.arange(c["tokens"])
        s["seq_ids"] = (at // c["len"]).to(torch.int32).to(dev)
        s["positions"] = (at % c["len"]).to(torch.int32).to(dev)
        shape = (c["tokens"], H, d)
        s["outs"] = [torch.empty(shape, dtype=DTYPES[c["out"]], device=dev) for _ in range(2)]
        if c["rope"]:
            angle = torch.arange(c["len"], dtype=torch.float64, device=dev)[:, None] * (
                ROPE_BASE ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=dev) / d))
            s["rope"] = torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()
    else:
        shape = (n_seqs, c["n_q"], c["heads"], d) if c["op"] == "chunk" else (n_seqs, c["heads"], d)
        s["Q"] = torch.randn(shape, generator=g, device=dev).to(DTYPES[c["q"]])
        s["lens"] = lens.to(torch.int32).to(dev)
        s["max_len"] = c["len_hi"]
        s["scale"] = 1.0 / math.sqrt(d)
        s["outs"] = [torch.empty(shape, dtype=DTYPES[c["out"]], device=dev)]
    if own:
        _handles(s)
    return s


def _handles(s):
    """The framework's own objects over the same memory."""
    import rotated_bit_kv_isoquant_b200 as iq
    c = s["case"]
    s["iq"] = iq
    s["params"] = iq.isoq_make_params(PARAM_SEED, c["d"], c["kv_heads"], bits=c["bits"])
    s["cache"] = iq.PagedCache(c["d"], c["kv_heads"], s["blocks"].shape[0], s["page_table"],
                               bits=c["bits"])
    s["cache"].blocks.copy_(s["blocks"])
    if c["op"] != "read":
        n = iq.isoq_window_workspace_bytes(c["n_seqs"], c["n_q"], c["heads"], c["kv_heads"], c["d"],
                                           s["max_len"], c["window"], c["sinks"])
        s["workspace"] = torch.empty((max(n, 16),), dtype=torch.uint8, device="cuda")


# ---- one pass ----------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    iq, c = s["iq"], s["case"]
    if c["op"] == "read":
        if c["rope"]:
            iq.isoq_dequantize_rope(s["params"], s["cache"], s["seq_ids"], s["positions"], *s["outs"],
                                    s["rope"])
        else:
            iq.isoq_dequantize(s["params"], s["cache"], s["seq_ids"], s["positions"], *s["outs"])
        return s["outs"]
    call = (iq.isoq_multi_token_attention_window if c["op"] == "chunk"
            else iq.isoq_decode_attention_window)
    call(s["params"], s["cache"], s["Q"], s["lens"], s["max_len"], c["window"], c["sinks"],
         s["outs"][0], s["scale"], s["workspace"])
    return s["outs"]


def _unpack_rows(w, bits):
    """int32 words [..., bits * d / 32] of one record -> table index [..., d]."""
    nib = 4 * torch.arange(8, device=w.device, dtype=torch.int32)
    if bits == 3:
        w = w.reshape(*w.shape[:-1], -1, 3)
        low = (w[..., None] >> nib) & 7
        top = (w[..., None] >> (nib + 3)) & 1
        spare = 4 * top[..., 0, :] + 2 * top[..., 1, :] + top[..., 2, :]
        return torch.cat([low, spare[..., None, :]], -2).flatten(-3)
    if bits == 4:
        return ((w[..., None] >> nib) & 15).flatten(-2)
    slots = 2 * torch.tensor(_slot2(), device=w.device, dtype=torch.int32)
    return ((w[..., None] >> slots) & 3).flatten(-2)


def _table(bits, dev):
    """The level of each unpacked value: 4-bit nibbles are sign and magnitude."""
    lev = MAGS[4] + [-m for m in MAGS[4]] if bits == 4 else _levels(bits)
    return torch.tensor(lev, device=dev)


def _fetch(s, seq, pos):
    """Rotated K and V [N..., H, d] of the tokens (seq, pos), norms over sqrt(d) included.
    Positions outside the kept pages read page 0 and are masked by the caller."""
    c = s["case"]
    d, H, bits = c["d"], c["kv_heads"], c["bits"]
    cw = bits * d // 32
    page = s["page_table"][seq, pos // PAGE].clamp(min=0).long()[..., None]
    slot = (pos % PAGE)[..., None, None]
    h = torch.arange(H, device=pos.device)
    words = s["blocks"].view(torch.int32)
    norms = s["blocks"].view(torch.float16)
    lev = _table(bits, pos.device)
    row = torch.arange(cw, device=pos.device)
    k = lev[_unpack_rows(words[page[..., None], h[:, None], slot * cw + row], bits)]
    v_at = PAGE * cw + PAGE // 2
    if bits == 3:
        u = torch.arange(d // 8, device=pos.device)[:, None]
        t, j = (slot >> 1) & 3, (slot & 1) | ((slot >> 2) & 2)
        group = (slot >> 4)[..., None] * (6 * d // 4) + ((u >> 1) * 8 + 2 * t[..., None] + (u & 1)) * 3
        w = words[page[..., None, None], h[:, None, None],
                  v_at + group + torch.arange(3, device=pos.device)]         # [..., H, d/8, 3]
        sh = (4 * j[..., None, None] + torch.tensor([0, 16], device=pos.device)).to(torch.int32)
        low = (w[..., None] >> sh) & 7
        top = (w[..., None] >> (sh + 3)) & 1
        spare = 4 * top[..., 0, :] + 2 * top[..., 1, :] + top[..., 2, :]
        v = lev[torch.cat([low, spare[..., None, :]], -2).flatten(-3)]
    else:
        v = lev[_unpack_rows(words[page[..., None], h[:, None], v_at + slot * cw + row], bits)]
    slot = slot[..., 0]
    kn = norms[page, h, 2 * PAGE * cw + slot].float() / math.sqrt(d)
    vn = norms[page, h, 4 * PAGE * cw + PAGE + slot].float() / math.sqrt(d)
    return k * kn[..., None], v * vn[..., None]


def _run_plain(s):
    c = s["case"]
    dt, R, dev = DTYPES[c["out"]], s["R"], s["R"].device
    if c["op"] == "read":
        k, v = _fetch(s, s["seq_ids"].long(), s["positions"].long())
        k, v = torch.einsum("nhe,hed->nhd", k, R), torch.einsum("nhe,hed->nhd", v, R)
        if c["rope"]:
            cs = s["rope"][s["positions"].long()][:, None]
            a, b = k.chunk(2, -1)
            k = torch.cat([a * cs[..., 0] + b * cs[..., 1], b * cs[..., 0] - a * cs[..., 1]], -1)
        return [k.to(dt), v.to(dt)]
    n, H, d, n_q = c["n_seqs"], c["kv_heads"], c["d"], c["n_q"]
    G = c["heads"] // H
    L = s["lens"].long()[:, None]
    W, S = min(c["window"], c["len_hi"]), min(c["sinks"], c["len_hi"])
    # the tokens that some query of the sequence may attend: the sinks, then the windows
    tail = L - (W + n_q - 1) + torch.arange(W + n_q - 1, device=dev)
    sink = torch.arange(S, device=dev).expand(n, S)
    pos = torch.cat([sink, tail], 1)                               # [n][T]
    at = L - n_q + torch.arange(n_q, device=dev)                   # query positions [n][n_q]
    in_tail = torch.arange(pos.shape[1], device=dev) >= S
    seen = (pos[:, None] <= at[..., None]) & (pos[:, None] >= 0) & torch.where(
        in_tail, (pos[:, None] > at[..., None] - W) & (pos[:, None] >= S), pos[:, None] < S)
    seq = torch.arange(n, device=dev)[:, None].expand_as(pos)
    reach = pos.clamp(min=0).minimum((L - 1).clamp(min=0))
    k, v = _fetch(s, seq, reach)                                   # [n][T][H][d]
    q = s["Q"].float().reshape(n, n_q, H, G, d)
    q = torch.einsum("nqhgd,hed->nhqge", q, R).reshape(n, H, n_q * G, d) * s["scale"]
    score = (q @ k.permute(0, 2, 3, 1)).reshape(n, H, n_q, G, -1)
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(score - top)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)               # rows that see nothing: zeros
    o = p.reshape(n, H, n_q * G, -1) @ v.permute(0, 2, 1, 3)
    o = torch.einsum("nhqge,hed->nqhgd", o.reshape(n, H, n_q, G, d), R)
    return [o.reshape(s["Q"].shape).to(dt)]


# ---- what a pass cannot do without -------------------------------------------------------
def work(case):
    c = case
    d, H = c["d"], c["kv_heads"]
    vec = c["bits"] * d // 8 + 2
    if c["op"] == "read":
        n = c["tokens"] * H * 2
        size = DTYPES[c["out"]].itemsize
        # WHT additions and the 4x4 blocks per vector
        return {"bytes": n * (vec + d * size) + 8 * c["tokens"],
                "flops": n * (d * math.log2(d) + 8 * d)}
    mean = (c["len_lo"] + c["len_hi"]) / 2
    kept = min(mean, c["window"] + c["n_q"] - 1 + c["sinks"])
    seen = min(mean, c["window"] + c["sinks"])
    rows = c["n_seqs"] * c["n_q"] * c["heads"]
    q = rows * d * (DTYPES[c["q"]].itemsize + DTYPES[c["out"]].itemsize)
    return {"bytes": c["n_seqs"] * kept * H * 2 * vec + q, "flops": 4.0 * d * rows * seen}


# ---- the definition in 64 bits -----------------------------------------------------------
def _bit_places(d, bits, side):
    """Bit offset in a page's K (side 0) or V (side 1) region of each bit of the field of
    (slot, dim): [64][d][bits], most significant first."""
    slot, dim, b = np.meshgrid(np.arange(PAGE), np.arange(d), np.arange(bits), indexing="ij")
    if bits == 4:
        return (slot * d + dim) * 4 + (3 - b)
    if bits == 2:
        return slot * 2 * d + (dim // 16) * 32 + 2 * np.array(_slot2())[dim % 16] + (1 - b)
    if side == 0:
        group, e = dim // 32, dim % 32
        word, nibble = e // 8, e % 8
        plain = (group * 3 + word) * 32 + 4 * nibble + (2 - b)
        spread = (group * 3 + b) * 32 + 4 * nibble + 3
        return slot * 3 * d + np.where(e < 24, plain, spread)
    block, t, j = slot // 16, (slot // 2) % 4, slot % 2 + 2 * (slot // 8 % 2)
    unit, e = dim // 8, dim % 8
    start = block * 48 * d + ((unit // 2) * 8 + 2 * t + unit % 2) * 96
    plain = start + (e // 2) * 32 + 4 * (j + 4 * (e % 2)) + (2 - b)
    spread = start + b * 32 + 4 * (j + 4 * (e % 2)) + 3
    return np.where(e < 6, plain, spread)


def _exact_pages(s):
    """K and V of every page as vectors [n_pages][64][H][d] in 64 bits."""
    c = s["case"]
    d, H, bits = c["d"], c["kv_heads"], c["bits"]
    dev, region = s["blocks"].device, PAGE * bits * d // 8
    R = torch.tensor(_rotation_of(d, H), device=dev)
    found = []
    for side in range(2):
        at = side * (region + 2 * PAGE)
        places = torch.tensor(_bit_places(d, bits, side).reshape(-1), device=dev)
        norm = s["blocks"][..., at + region:at + region + 2 * PAGE].contiguous().view(torch.float16)
        whole = []
        for p in range(0, s["blocks"].shape[0], 256):
            codes = s["blocks"][p:p + 256, :, at:at + region]
            raw = (codes[..., places // 8] >> (places % 8)) & 1
            weight = torch.tensor([2 ** (bits - 1 - b) for b in range(bits)], device=dev)
            field = (raw.reshape(-1, H, PAGE, d, bits).long() * weight).sum(-1)
            mag = torch.tensor(MAGS[bits], dtype=torch.float64, device=dev)
            if bits == 4:
                level = mag[field % 8] * torch.where(field >= 8, -1.0, 1.0).double()
            else:
                half = 2 ** (bits - 1)
                level = torch.where(field >= half, mag[(field - half).clamp(min=0)],
                                    -mag[(half - 1 - field).clamp(min=0)])
            z = level * (norm[p:p + 256].double() / math.sqrt(d))[..., None]
            whole.append((z @ R).transpose(1, 2))                  # x = R^T z
        found.append(torch.cat(whole))
    return found


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    K, V = _exact_pages(s)
    dt = torch.float64
    if c["op"] == "read":
        pos = s["positions"].long()
        page = s["page_table"][s["seq_ids"].long(), pos // PAGE].long()
        k, v = K[page, pos % PAGE], V[page, pos % PAGE]
        if c["rope"]:
            half = c["d"] // 2
            angle = pos.to(dt)[:, None] * ROPE_BASE ** (
                -torch.arange(half, dtype=dt, device=pos.device) / half)
            turn = torch.polar(torch.ones_like(angle), -angle)[:, None]
            turned = torch.complex(k[..., :half], k[..., half:]) * turn
            k = torch.cat([turned.real, turned.imag], -1)
        return [k, v]
    n_q, G = c["n_q"], c["heads"] // c["kv_heads"]
    Q = s["Q"].to(dt).reshape(c["n_seqs"], n_q, c["kv_heads"], G, c["d"])
    out = torch.zeros_like(Q)
    for i, L in enumerate(s["lens"].tolist()):
        lo = max(0, L - n_q + 1 - c["window"])
        pos = [t for t in range(min(c["sinks"], L)) if t < lo] + list(range(lo, L))
        if not pos:
            continue
        pos = torch.tensor(pos, device=Q.device)
        page = s["page_table"][i, pos // PAGE].long()
        k, v = K[page, pos % PAGE], V[page, pos % PAGE]            # [T][H][d]
        at = (L - n_q + torch.arange(n_q, device=Q.device))[:, None]
        hidden = (pos > at) | ((pos <= at - c["window"]) & (pos >= c["sinks"]))
        for h in range(c["kv_heads"]):
            x = torch.einsum("qgd,td->qgt", Q[i, :, h], k[:, h]) / math.sqrt(c["d"])
            x = x.masked_fill(hidden[:, None], -math.inf)
            some = ~hidden.all(-1)
            out[i, some, h] = torch.softmax(x[some], -1) @ v[:, h]
    return [out.reshape(s["Q"].shape)]
