"""The operators around the attention as measured: their cases, their plain forms and the library's calls.

* ``rope``: rotary positions applied to (or, ``inverse``, taken off) part of every head;
* ``norm_rope``: RMS norm of every head of q and k and the rotation, in one pass;
* ``kv_append``: new tokens' K rows, normalised and rotated on the way, and V rows into the paged pool;
* ``latent_append``: the same for rows [c | r] of the latent cache (c normalised, r rotated);
* ``tree``: latent attention of the drafted tokens of a tree, behind the context of their sequence.

A rotary table is ``turns``: the frequencies in turns a position, as 64-bit binary fractions.
"""
import math

import numpy as np
import torch

own = False

L, R = 512, 64            # latent and rotary widths of the latent cache
EPS = 1e-6


def listed():
    return [
        # one decoding step of 8 sequences: the rotation taken off the attention's output (latency)
        {"name": "rope_back_t8", "op": "rope", "tokens": 8, "heads": 64, "dim": 512, "rot": 64, "wide": 512,
         "half": False, "inverse": True, "yarn": 1.0, "far": 32768},
        # a prompt chunk's rotary queries out of the query projection (heads of 192 values), long context
        {"name": "rope_view_t8192", "op": "rope", "tokens": 8192, "heads": 64, "dim": 64, "rot": 64, "wide": 192,
         "half": False, "inverse": False, "yarn": 32.0, "far": 131072},
        # one token; a prompt of the benchmark's length; grouped heads, every value rotated, an odd length
        {"name": "norm_rope_t1", "op": "norm_rope", "tokens": 1, "heads": 64, "kheads": 1, "dim": 512, "rot": 64,
         "half": False, "yarn": 1.0, "far": 32768, "w32": False},
        {"name": "norm_rope_t8192", "op": "norm_rope", "tokens": 8192, "heads": 64, "kheads": 1, "dim": 512,
         "rot": 64, "half": False, "yarn": 16.0, "far": 65536, "w32": False},
        {"name": "norm_rope_gqa_t3001", "op": "norm_rope", "tokens": 3001, "heads": 20, "kheads": 4, "dim": 128,
         "rot": 128, "half": True, "yarn": 1.0, "far": 8192, "w32": True},
        # one decoding step's new rows of 8 sequences (latency), and a long prompt's in one call
        {"name": "kv_append_fp8_t8", "op": "kv_append", "fp8": True, "tokens": 8, "seqs": 8, "page": 64,
         "dim": 512, "rot": 64, "half": False, "yarn": 1.0, "far": 32768, "norm": True},
        {"name": "kv_append_bf16_t65536", "op": "kv_append", "fp8": False, "tokens": 65536, "seqs": 3, "page": 64,
         "dim": 512, "rot": 64, "half": False, "yarn": 16.0, "far": 65536, "norm": True},
        {"name": "latent_append_bf16_t777", "op": "latent_append", "fp8": False, "tokens": 777, "seqs": 5,
         "page": 24, "half": True, "yarn": 1.0, "far": 4096},
        {"name": "latent_append_fp8_t65536", "op": "latent_append", "fp8": True, "tokens": 65536, "seqs": 3,
         "page": 64, "half": False, "yarn": 32.0, "far": 131072},
        # one user's draft of 8 tokens (latency); a batch of drafts, all heads; large trees on few heads
        {"name": "tree_bf16_b1_n8", "op": "tree", "fp8": False, "seqs": 1, "n_lo": 8, "n_hi": 8, "heads": 64,
         "lo": 4097, "hi": 4097, "lens": 1, "page": 64},
        {"name": "tree_bf16_b32_n16", "op": "tree", "fp8": False, "seqs": 32, "n_lo": 5, "n_hi": 16, "heads": 128,
         "lo": 100, "hi": 8192, "lens": 2, "page": 64},
        {"name": "tree_fp8_b12_n60", "op": "tree", "fp8": True, "seqs": 12, "n_lo": 20, "n_hi": 60, "heads": 16,
         "lo": 1, "hi": 20000, "lens": 3, "page": 24},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "kv_append", "latent_append", "tree", "tree", "tree"])
    half, fp8 = rng.random() < 0.5, rng.random() < 0.5
    far = {"half": half, "yarn": rng.choice([1.0, 8.0, 32.0]), "far": _log_int(rng, 1000, 1000000)}
    page = rng.choice([16, 24, 32, 64, 128])
    if op in ("rope", "norm_rope"):
        dim = rng.choice([64, 128, 192, 512])
        heads = rng.choice([1, 8, 20, 64, 128])
        case = {"op": op, "tokens": _log_int(rng, 1, min(65536, 8192 * 64 * 512 // (heads * dim))),
                "heads": heads, "dim": dim, "rot": rng.choice([32, 64, dim if dim < 256 else 64]), **far}
        if op == "rope":
            return {**case, "wide": dim + rng.choice([0, 64, 128]), "inverse": rng.random() < 0.5}
        return {**case, "kheads": rng.choice([1, 2, 8]), "w32": rng.random() < 0.5}
    if op in ("kv_append", "latent_append"):
        case = {"op": op, "fp8": fp8, "tokens": _log_int(rng, 1, 65000), "seqs": rng.randint(1, 8), "page": page,
                **far}
        if op == "kv_append":
            case.update(dim=rng.choice([64, 128, 512]), rot=rng.choice([32, 64]), norm=rng.random() < 0.7)
        return case
    n_hi, heads = rng.choice([1, 3, 8, 16, 33, 64]), rng.choice([16, 20, 64, 128])
    most = 170000000 // (n_hi * heads)                # entries that all sequences may have
    hi = _log_int(rng, 50, min(60000, most))
    seqs = _log_int(rng, 1, min(40, most // hi))
    return {"op": "tree", "fp8": fp8, "seqs": seqs, "n_lo": rng.randint(1, n_hi), "n_hi": n_hi, "heads": heads,
            "lo": rng.randint(0, hi), "hi": hi, "lens": rng.randrange(1 << 30), "page": page}


def _lengths(case):
    """Context lengths and numbers of drafted tokens of a tree case: part of the case."""
    r = np.random.RandomState(case["lens"] % (1 << 32))
    return (r.randint(case["lo"], case["hi"] + 1, case["seqs"]),
            r.randint(case["n_lo"], case["n_hi"] + 1, case["seqs"]))


def _frequencies(rot, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Frequencies (radians a position) in 64 bits: plain, or interpolated where a pair turns less than
    `fast` times within the original length (all the way where it turns less than `slow` times)."""
    i = np.arange(0, rot, 2, dtype=np.float64)
    f = base ** (-i / rot)
    if factor == 1.0:
        return f, 1.0
    at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot // 2 - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _pages(g, lens, page):
    """Random physical pages for every sequence, some to spare: (number of blocks, block table)."""
    need = [max(1, -(-int(n) // page)) for n in lens]
    blocks = sum(need) + 3
    perm = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return blocks, table


def _codes(y):
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _quantise(x, low):
    """e4m3 rows of fp32 rows x [n, W]: codes (the last `low` values as a high and a low code), scales."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    y = x / scale[:, None]
    hi = _codes(y)
    if not low:
        return hi.view(torch.uint8), scale
    rest = _codes(y[:, -low:] - hi[:, -low:].float())
    return torch.cat([hi.view(torch.uint8), rest.view(torch.uint8)], 1), scale


def _dequantise(codes, scale):
    """fp32 rows [..., L + R] of codes [..., L + 2R] (uint8) and scales [...]."""
    v = codes.view(torch.float8_e4m3fn).float()
    return torch.cat([v[..., :L], v[..., L:L + R] + v[..., L + R:]], -1) * scale[..., None]


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _weight(g, n, dtype):
    return (1.0 + 0.2 * _normal(g, n)).to(dtype)


def _prepare_tree(case, s, g, seed):
    """Contexts and drafted tokens of the sequences; a drafted token follows any earlier one, or the context."""
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, n = _lengths(case)
    r, words = np.random.RandomState(seed % (1 << 32)), -(-int(n.max()) // 32)
    mask = np.zeros((int(n.sum()), words), dtype=np.uint32)
    row = 0
    for k in n:
        for i in range(k):
            parent = r.randint(-1, i) if i else -1
            if parent >= 0:
                mask[row + i] = mask[row + parent]
            mask[row + i, i // 32] |= np.uint32(1 << (i % 32))
        row += k
    T, H = row, case["heads"]
    s.update(context_lens=torch.tensor(ctx, **i32), cu_tokens=torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32),
             tree_mask=torch.from_numpy(mask.view(np.int32)).cuda(), max_n=int(n.max()), max_len=int((ctx + n).max()),
             q_latent=_normal(g, T, H, L).to(torch.bfloat16), q_rope=_normal(g, T, H, R).to(torch.bfloat16),
             scale=(128 + R) ** -0.5)
    blocks, s["block_table"] = _pages(g, ctx + n, case["page"])
    rows = _normal(g, blocks * case["page"], L + R)
    rows[:, L:] *= 3.0
    rows = rows.to(torch.bfloat16)
    if s["fp8"]:
        codes, s["pool_scale"] = _quantise(rows.float(), R)
        s["rows"] = codes.view(blocks, case["page"], L + 2 * R)
    else:
        s["rows"] = rows.view(blocks, case["page"], L + R)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    op, bf16 = case["op"], torch.bfloat16
    s = {"op": op, "fp8": case.get("fp8", False)}
    if op == "tree":
        _prepare_tree(case, s, g, seed)
        return s
    T = case["tokens"]
    f, s["amplitude"] = _frequencies(case.get("rot", R), case["yarn"])
    s["half"], s["inverse"] = case["half"], case.get("inverse", False)
    s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    s["turns"] = torch.tensor(np.round(f / (2 * math.pi) * 2.0 ** 64).astype(np.int64), device="cuda")
    if op in ("rope", "norm_rope"):
        # a stretch of a long document (or the last tokens of several), ending at the furthest position
        s["positions"] = (torch.arange(T, **i32) + max(0, case["far"] - T))
        H, D = case["heads"], case["dim"]
        if op == "rope":
            s["x"] = _normal(g, T, H, case["wide"]).to(bf16)[..., case["wide"] - D:]
        else:
            w = torch.float32 if case["w32"] else bf16
            qk = (3.0 * _normal(g, T, (H + case["kheads"]) * D)).to(bf16)     # one projection's output
            s["q"], s["k"] = (t.unflatten(1, (-1, D)) for t in (qk[:, :H * D], qk[:, H * D:]))
            s["q_weight"], s["k_weight"] = _weight(g, D, w), _weight(g, D, w)
        return s
    # appending: the rows of each sequence follow what it has, at far positions but in a cache of these only
    lens = [T * (b + 1) // case["seqs"] - T * b // case["seqs"] for b in range(case["seqs"])]
    s["seq_of_token"] = torch.cat([torch.full((n,), b, **i32) for b, n in enumerate(lens)])
    s["entries"] = torch.cat([torch.arange(11, 11 + n, **i32) for n in lens])
    s["positions"] = s["entries"] + max(0, case["far"] - max(lens) - 11)
    blocks, s["block_table"] = _pages(g, [n + 11 for n in lens], case["page"])
    s["eps"] = EPS if case.get("norm", True) else None
    if op == "kv_append":
        D = case["dim"]
        s["k"], s["v"] = (3.0 * _normal(g, T, D)).to(bf16), _normal(g, T, D).to(bf16)
        s["weight"] = _weight(g, D, bf16) if case["norm"] else None
        old = _normal(g, blocks * case["page"] * 2, D).to(bf16)
        if s["fp8"]:
            codes, scale = _quantise(old.float(), 0)
            s["k_scale"], s["v_scale"] = scale.view(-1, 2).t().contiguous()
            old = codes
        s["kv"] = old.view(blocks, case["page"], 2, D)
        return s
    x = (3.0 * _normal(g, T, L + R)).to(bf16)                                 # one projection's output
    s["latent"], s["rope"], s["weight"] = x[:, :L], x[:, L:], _weight(g, L, bf16)
    old = _normal(g, blocks * case["page"], L + R).to(bf16)
    if s["fp8"]:
        codes, s["pool_scale"] = _quantise(old.float(), R)
        s["rows"] = codes.view(blocks, case["page"], L + 2 * R)
    else:
        s["rows"] = old.view(blocks, case["page"], L + R)
    return s


# ---- plain forms ----------------------------------------------------------------------------
def _rotate(s, x, last):
    """fp32 x [T, .., D], its last values rotated by the tokens' angles (worked out in 64 bits)."""
    angle = s["positions"].double()[:, None] * s["freq"]
    angle = angle.view(angle.shape[:1] + (1,) * (x.dim() - 2) + angle.shape[1:])
    m = s["amplitude"]
    c, z = (angle.cos() * m).float(), (angle.sin() * (-m if s["inverse"] else m)).float()
    p = x[..., x.shape[-1] - last:]
    if s["half"]:
        a, b = p[..., :last // 2], p[..., last // 2:]
        p = torch.cat([a * c - b * z, b * c + a * z], -1)
    else:
        a, b = p[..., 0::2], p[..., 1::2]
        p = torch.stack([a * c - b * z, b * c + a * z], -1).flatten(-2)
    return torch.cat([x[..., :x.shape[-1] - last], p], -1)


def _norm(x, weight, eps):
    x = x.float()
    if eps is None:
        return x
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return y if weight is None else y * weight.float()


def _slots(s, page):
    x = s["entries"].long()
    return s["block_table"][s["seq_of_token"].long(), x // page].long() * page + x % page


def _kv_append_plain(s, rot):
    at = _slots(s, s["kv"].shape[1])
    kv = s["kv"].view(-1, 2, s["kv"].shape[3])
    k, v = _rotate(s, _norm(s["k"], s["weight"], s["eps"]), rot), s["v"].float()
    if s["fp8"]:
        kv[at, 0], s["k_scale"][at] = _quantise(k, 0)
        kv[at, 1], s["v_scale"][at] = _quantise(v, 0)
    else:
        kv[at, 0], kv[at, 1] = k.to(kv.dtype), v.to(kv.dtype)


def _latent_append_plain(s):
    at = _slots(s, s["rows"].shape[1])
    rows = s["rows"].view(-1, s["rows"].shape[2])
    x = torch.cat([_norm(s["latent"], s["weight"], s["eps"]), _rotate(s, s["rope"].float(), R)], 1)
    if s["fp8"]:
        rows[at], s["pool_scale"][at] = _quantise(x, R)
    else:
        rows[at] = x.to(rows.dtype)


def _tree_plain(s):
    cu, ctx = s["cu_tokens"].long(), s["context_lens"].long()
    T, H, B, page = s["q_latent"].shape[0], s["q_latent"].shape[1], ctx.numel(), s["rows"].shape[1]
    i, j = torch.arange(s["max_n"], device="cuda"), torch.arange(s["max_len"], device="cuda")
    n = cu[1:] - cu[:-1]
    tok = (cu[:-1, None] + i).clamp_max(T - 1)                              # [B, n]
    draft = j - ctx[:, None]                                                # [B, k]
    known = (draft >= 0) & (draft < n[:, None])
    word = torch.where(known, draft, 0) // 32
    bits = torch.gather(s["tree_mask"][tok], 2, word[:, None].expand(-1, i.numel(), -1))
    seen = (draft < 0)[:, None] | (known[:, None] & ((bits >> (draft % 32)[:, None]) & 1).bool())
    exists = draft < n[:, None]
    at = s["block_table"][torch.arange(B, device="cuda")[:, None], torch.where(exists, j, 0) // page].long() * page \
        + torch.where(exists, j, 0) % page
    rows = s["rows"].view(-1, s["rows"].shape[2])[at]                       # [B, k, width]
    x = _dequantise(rows, s["pool_scale"][at]) if s["fp8"] else rows.float()
    q = torch.cat([s["q_latent"], s["q_rope"]], -1)[tok].float()            # [B, n, H, L + R]
    score = torch.matmul(q.flatten(1, 2), x.transpose(1, 2)).view(B, i.numel(), H, -1)
    score.mul_(s["scale"]).masked_fill_(~seen[:, :, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    out = torch.matmul(score.flatten(1, 2), x[..., :L]).view(B, i.numel(), H, L)
    out = out / score.sum(-1, keepdim=True).clamp_min(1e-30)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp_max(B - 1)
    return out[b, t - cu[b]].to(torch.bfloat16)


def _run_plain(s):
    if s["op"] == "rope":
        return _rotate(s, s["x"].float(), 2 * s["freq"].numel()).to(torch.bfloat16)
    if s["op"] == "norm_rope":
        q, k = _norm(s["q"], s["q_weight"], EPS), _norm(s["k"], s["k_weight"], EPS)
        rot = 2 * s["freq"].numel()
        return _rotate(s, q, rot).to(torch.bfloat16), _rotate(s, k, rot).to(torch.bfloat16)
    if s["op"] == "tree":
        return _tree_plain(s)
    _kv_append_plain(s, 2 * s["freq"].numel()) if s["op"] == "kv_append" else _latent_append_plain(s)
    return _appended(s)


def _appended(s):
    kind = torch.float8_e4m3fn if s["fp8"] else torch.bfloat16
    if s["op"] == "kv_append":
        out = {"kv": s["kv"].view(kind)}
        return {**out, "k_scale": s["k_scale"], "v_scale": s["v_scale"]} if s["fp8"] else out
    out = {"rows": s["rows"].view(kind)}
    return {**out, "scale": s["pool_scale"]} if s["fp8"] else out


def _run_own(s):
    import sparse_paged_attention_gb300 as spa
    op, fp8 = s["op"], s["fp8"]
    if op == "tree":
        pool = spa.LatentPool(s["rows"], s["block_table"], R, s["pool_scale"] if fp8 else None)
        f = spa.sparse_attn_latent_tree_decode_fp8 if fp8 else spa.sparse_attn_latent_tree_decode
        return f(s["q_latent"], s["q_rope"], pool, s["context_lens"], s["cu_tokens"], s["tree_mask"],
                 scale=s["scale"])
    table = spa.RotaryTable(s["turns"], not s["half"], s["amplitude"])
    if op == "rope":
        return spa.sparse_attn_rope(s["x"], s["positions"], table, inverse=s["inverse"])
    if op == "norm_rope":
        return spa.sparse_attn_norm_rope(s["q"], s["k"], s["positions"], table, q_weight=s["q_weight"],
                                         k_weight=s["k_weight"], eps=EPS)
    kw = dict(weight=s["weight"], eps=s["eps"], entries=s["entries"], seq_of_token=s["seq_of_token"])
    if op == "kv_append":
        pool = spa.PagedPool(s["kv"], s["block_table"], s.get("k_scale"), s.get("v_scale"))
        f = spa.sparse_attn_paged_kv_append_fp8 if fp8 else spa.sparse_attn_paged_kv_append
        f(s["k"], s["v"], s["positions"], pool, table, **kw)
    else:
        pool = spa.LatentPool(s["rows"], s["block_table"], R, s.get("pool_scale"))
        f = spa.sparse_attn_latent_append_fp8 if fp8 else spa.sparse_attn_latent_append
        f(s["latent"], s["rope"], s["positions"], pool, table, **kw)
    return _appended(s)


def run(s):
    return _run_own(s) if own else _run_plain(s)


def work(case):
    op = case["op"]
    if op == "tree":
        ctx, n = (x.astype(np.int64) for x in _lengths(case))
        H, T = case["heads"], float(n.sum())
        row = L + 2 * R + 4 if case["fp8"] else 2 * (L + R)
        # (a token sees its sequence's context and, of the tree, its ancestors: at least itself)
        return {"bytes": float((ctx + n).sum()) * row + 2.0 * T * H * (2 * L + R),
                "flops": 2.0 * H * (2 * L + R) * float((n * (ctx + 1)).sum())}
    T = float(case["tokens"])
    if op in ("rope", "norm_rope"):
        heads = case["heads"] + case.get("kheads", 0)
        return {"bytes": 4.0 * T * heads * case["dim"] + 4.0 * T, "flops": 0.0}
    width = 2 * case["dim"] if op == "kv_append" else L + R
    out = width + (8.0 if op == "kv_append" else R + 4.0) if case["fp8"] else 2.0 * width
    return {"bytes": T * (2.0 * width + out + 12), "flops": 0.0}


# ---- the definitions in 64 bits -------------------------------------------------------------
def _turned(s, x):
    """x [.., W] in 64 bits, all of it pairs, by complex multiplication."""
    pos = s["positions"].double()
    turn = torch.polar(torch.full_like(pos, s["amplitude"])[:, None].expand(-1, s["freq"].numel()).contiguous(),
                       pos[:, None] * s["freq"] * (-1.0 if s["inverse"] else 1.0))
    for _ in range(x.dim() - 2):
        turn = turn.unsqueeze(1)
    if s["half"]:
        h = x.shape[-1] // 2
        y = torch.complex(x[..., :h], x[..., h:]) * turn
        return torch.cat([y.real, y.imag], -1)
    y = torch.view_as_complex(x.reshape(x.shape[:-1] + (-1, 2)).contiguous()) * turn
    return torch.view_as_real(y).reshape(x.shape)


def _row64(s, x, weight, eps, rot):
    x = x.double()
    if eps is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt()
        if weight is not None:
            x = x * weight.double()
    keep = x.shape[-1] - rot
    return torch.cat([x[..., :keep], _turned(s, x[..., keep:])], -1) if rot else x


def _values64(s):
    """The latent cache's rows in 64 bits, [rows, L + R]."""
    rows = s["rows"].reshape(-1, s["rows"].shape[2])
    if not s["fp8"]:
        return rows.double()
    v = rows.view(torch.float8_e4m3fn).double()
    v[:, L:L + R] += v[:, L + R:]
    return v[:, :L + R] * s["pool_scale"].double()[:, None]


def _exact_tree(case, s):
    rows, table, page = _values64(s), s["block_table"].tolist(), case["page"]
    cu, ctx, mask = s["cu_tokens"].tolist(), s["context_lens"].tolist(), s["tree_mask"].cpu().numpy().view(np.uint32)
    outs = []
    for b in range(case["seqs"]):
        n, end = cu[b + 1] - cu[b], ctx[b] + cu[b + 1] - cu[b]
        at = torch.tensor([table[b][p] for p in range(-(-end // page))], device="cuda") * page
        x = rows[(at[:, None] + torch.arange(page, device="cuda")).reshape(-1)[:end]]
        for t in range(cu[b], cu[b + 1]):
            see = list(range(ctx[b])) + [ctx[b] + i for i in range(n) if mask[t, i // 32] >> (i % 32) & 1]
            y = x[torch.tensor(see, device="cuda")]
            z = s["q_latent"][t].double() @ y[:, :L].T + s["q_rope"][t].double() @ y[:, L:].T
            outs.append(torch.softmax(z * s["scale"], dim=-1) @ y[:, :L])
    return torch.stack(outs)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tree":
        # (64-bit products take some milliseconds a token where sequences are long)
        ctx, n = _lengths(case)
        return _exact_tree(case, s) if float((n * (ctx + n)).sum()) * case["heads"] < 4e8 else None
    if op == "rope":
        return _row64(s, s["x"], None, None, case["rot"])
    if op == "norm_rope":
        return tuple(_row64(s, s[x], s[x + "_weight"], EPS, case["rot"]) for x in ("q", "k"))
    page = case["page"]
    table = s["block_table"].cpu().numpy()
    e, b = s["entries"].cpu().numpy(), s["seq_of_token"].cpu().numpy()
    at = torch.from_numpy(table[b, e // page].astype(np.int64) * page + e % page).cuda()
    if op == "kv_append":
        kv = s["kv"].view(torch.float8_e4m3fn).double() if s["fp8"] else s["kv"].double()
        flat = kv.view(-1, 2, case["dim"])
        new = torch.stack([_row64(s, s["k"], s["weight"], s["eps"], case["rot"]), s["v"].double()], 1)
        if not s["fp8"]:
            flat[at] = new
            return {"kv": kv}
        unit = new.abs().amax(-1) / 448.0
        flat[at] = new / unit[..., None]
        scale = torch.stack([s["k_scale"], s["v_scale"]], 1).double()
        scale[at] = unit
        return {"kv": kv, "k_scale": scale[:, 0].contiguous(), "v_scale": scale[:, 1].contiguous()}
    new = torch.cat([_row64(s, s["latent"], s["weight"], s["eps"], 0), _turned(s, s["rope"].double())], 1)
    if not s["fp8"]:
        rows = s["rows"].double()
        rows.view(-1, L + R)[at] = new
        return {"rows": rows}
    rows, scale = s["rows"].view(torch.float8_e4m3fn).double(), s["pool_scale"].double()
    scale[at] = new.abs().amax(1) / 448.0
    y = new / scale[at][:, None]
    low = y[:, L:] - y[:, L:].float().to(torch.float8_e4m3fn).double()
    rows.view(-1, L + 2 * R)[at] = torch.cat([y, low], 1)
    return {"rows": rows, "scale": scale}
