"""The latent-attention operators as measured: their cases, their plain forms and the library's calls.

Latent attention keeps ONE vector a token in the paged cache, a latent part of L values (key and value
at once) and a rotary part of R values (key only).  Five operators:

* ``write``: new tokens' rows go to their pool slots, copied (bf16) or quantised to e4m3 with one
  scale a row (the rotary part as two codes a value, high and low);
* ``read``: rows of the cache back as bf16;
* ``decode``: the absorbed form, queries against the cached latents, one token or a few a sequence;
* ``prefill``: the expanded form, per-head keys and values of ragged causal sequences.
"""
import math

import numpy as np
import torch

own = False

L, R = 512, 64            # latent and rotary widths: the library's head_dim, and one 128-byte chunk
DN, DR, DV = 128, 64, 128  # expanded form: widths of the plain key, the rotary key and the value


def listed():
    return [
        # one decoding step's new rows of 8 sequences: latency
        {"name": "write_fp8_t8", "op": "write", "fp8": True, "tokens": 8, "seqs": 8, "page": 64},
        # a long prompt's rows in one call: memory rate (the KV write's benchmark length)
        {"name": "write_fp8_t65536", "op": "write", "fp8": True, "tokens": 65536, "seqs": 3, "page": 64},
        {"name": "write_bf16_t30001", "op": "write", "fp8": False, "tokens": 30001, "seqs": 5, "page": 24},
        # a short prefix and a long one brought back for the expanded form
        {"name": "read_fp8_t777", "op": "read", "fp8": True, "tokens": 777, "seqs": 2, "page": 24},
        {"name": "read_fp8_t65536", "op": "read", "fp8": True, "tokens": 65536, "seqs": 4, "page": 64},
        # one user, a short context: latency; then batches of ragged contexts
        {"name": "decode_bf16_b1_4k", "op": "decode", "fp8": False, "seqs": 1, "q": 1, "heads": 64,
         "lo": 4097, "hi": 4097, "lens": 1, "page": 64},
        {"name": "decode_bf16_b64_16k", "op": "decode", "fp8": False, "seqs": 64, "q": 1, "heads": 128,
         "lo": 100, "hi": 16384, "lens": 2, "page": 64},
        # two tokens a sequence (a drafted token checked), e4m3 rows
        {"name": "decode_fp8_b48_q2", "op": "decode", "fp8": True, "seqs": 48, "q": 2, "heads": 64,
         "lo": 1, "hi": 12000, "lens": 3, "page": 64},
        # one very long context, few heads, pages that end inside a tile
        {"name": "decode_fp8_b1_128k", "op": "decode", "fp8": True, "seqs": 1, "q": 1, "heads": 16,
         "lo": 131071, "hi": 131071, "lens": 4, "page": 24},
        # short ragged prompts; one long prompt; a chunk after a long cached prefix
        {"name": "prefill_b5_short", "op": "prefill", "seqs": 5, "heads": 16, "lo": 1, "hi": 300,
         "prefix": 0, "lens": 5},
        {"name": "prefill_b1_8k", "op": "prefill", "seqs": 1, "heads": 64, "lo": 8192, "hi": 8192,
         "prefix": 0, "lens": 6},
        {"name": "prefill_b2_1k_after_12k", "op": "prefill", "seqs": 2, "heads": 64, "lo": 900,
         "hi": 1100, "prefix": 12000, "lens": 7},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prefill", "prefill"])
    fp8 = rng.random() < 0.5
    page = rng.choice([16, 24, 32, 64, 128])
    lens = rng.randrange(1 << 30)
    if op in ("write", "read"):
        return {"op": op, "fp8": fp8, "tokens": _log_int(rng, 8, 65000), "seqs": rng.randint(1, 8),
                "page": page}
    if op == "decode":
        hi = _log_int(rng, 100, 100000)
        q = rng.choice([1, 1, 2, 3])
        seqs = _log_int(rng, 1, max(1, min(64, 400000 // (hi * q))))
        return {"op": op, "fp8": fp8, "seqs": seqs, "q": q, "heads": rng.choice([16, 20, 64, 128]),
                "lo": rng.randint(1, hi), "hi": hi, "lens": lens, "page": page}
    hi = _log_int(rng, 20, 4000)
    prefix = rng.choice([0, 0, _log_int(rng, 10, 8000)])
    seqs = rng.randint(1, max(1, min(6, 24000000 // (hi * (hi + prefix)))))
    return {"op": op, "seqs": seqs, "heads": rng.choice([16, 20, 64]), "lo": rng.randint(1, hi),
            "hi": hi, "prefix": prefix, "lens": lens}


def _lengths(case):
    """New tokens (prefill) or context lengths (decode) of the sequences: part of the case."""
    return np.random.RandomState(case["lens"] % (1 << 32)).randint(case["lo"], case["hi"] + 1,
                                                                   case["seqs"])


def _split(tokens, seqs):
    """The tokens of a write or read dealt to its sequences."""
    return [tokens * (b + 1) // seqs - tokens * b // seqs for b in range(seqs)]


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


def _quantise(x):
    """e4m3 rows of fp32 rows x [n, L + R]: codes [n, L + 2R] as float8, scales [n]."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    y = x / scale[:, None]
    hi = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    lo = (y[:, L:] - hi[:, L:].float()).to(torch.float8_e4m3fn)
    return torch.cat([hi.view(torch.uint8), lo.view(torch.uint8)], 1), scale


def _dequantise(codes, scale):
    """fp32 rows [..., L + R] of codes [..., L + 2R] (uint8) and scales [...]."""
    v = codes.view(torch.float8_e4m3fn).float()
    return torch.cat([v[..., :L], v[..., L:L + R] + v[..., L + R:]], -1) * scale[..., None]


def _randn_rows(g, n):
    """Rows as a cache holds them: a normalised latent, a rotary part a few times larger."""
    x = torch.randn((n, L + R), generator=g, device="cuda")
    x[:, L:] *= 3.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"op": case["op"], "fp8": case.get("fp8", False)}
    if case["op"] == "prefill":
        lens, prefix, H = _lengths(case), case["prefix"], case["heads"]
        klens = lens + prefix
        T, S = int(lens.sum()), int(klens.sum())
        q = torch.randn((T, H, DN + DR), generator=g, device="cuda").to(torch.bfloat16)
        kv = torch.randn((S, H, DN + DV), generator=g, device="cuda").to(torch.bfloat16)
        s.update(q=q, k_nope=kv[..., :DN], v=kv[..., DN:],
                 k_rope=torch.randn((S, DR), generator=g, device="cuda").to(torch.bfloat16),
                 cu_q=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), **i32),
                 cu_k=torch.tensor(np.concatenate([[0], np.cumsum(klens)]), **i32),
                 max_q=int(lens.max()), max_k=int(klens.max()), scale=(DN + DR) ** -0.5)
        return s
    if case["op"] == "decode":
        lens = _lengths(case)
        n = case["q"]
        s["seq_of_token"] = torch.arange(case["seqs"], **i32).repeat_interleave(n)
        last = torch.tensor(lens - 1, **i32).repeat_interleave(n)
        back = torch.arange(n - 1, -1, -1, **i32).repeat(case["seqs"])
        s["positions"] = (last - back).clamp_min(0)
        T, H = case["seqs"] * n, case["heads"]
        s["q_latent"] = torch.randn((T, H, L), generator=g, device="cuda").to(torch.bfloat16)
        s["q_rope"] = torch.randn((T, H, R), generator=g, device="cuda").to(torch.bfloat16)
        s["max_len"] = int(lens.max())
        s["scale"] = (DN + DR) ** -0.5
    else:
        lens = _split(case["tokens"], case["seqs"])
        first = 11            # the rows of each sequence start after a few older ones
        s["seq_of_token"] = torch.cat([torch.full((n,), b, **i32) for b, n in enumerate(lens)])
        s["positions"] = torch.cat([torch.arange(first, first + n, **i32) for n in lens])
        lens = [n + first for n in lens]
    blocks, s["block_table"] = _pages(g, lens, case["page"])
    rows = _randn_rows(g, blocks * case["page"])
    if s["fp8"]:
        codes, s["pool_scale"] = _quantise(rows.float())
        s["rows"] = codes.view(blocks, case["page"], L + 2 * R)
    else:
        s["rows"] = rows.view(blocks, case["page"], L + R)
    if case["op"] == "write":
        new = _randn_rows(g, case["tokens"])
        s["latent"], s["rope"] = new[:, :L].contiguous(), new[:, L:].contiguous()
    return s


def _slots(s, b, x):
    """Pool rows of positions x of sequences b."""
    page = s["rows"].shape[1]
    return s["block_table"][b, x // page].long() * page + x % page


def _write_plain(s):
    at = _slots(s, s["seq_of_token"].long(), s["positions"].long())
    rows = s["rows"].view(-1, s["rows"].shape[2])
    x = torch.cat([s["latent"], s["rope"]], 1)
    if s["fp8"]:
        rows[at], s["pool_scale"][at] = _quantise(x.float())
    else:
        rows[at] = x


def _read_plain(s):
    at = _slots(s, s["seq_of_token"].long(), s["positions"].long())
    rows = s["rows"].view(-1, s["rows"].shape[2])[at]
    return _dequantise(rows, s["pool_scale"][at]).to(torch.bfloat16) if s["fp8"] else rows


def _decode_plain(s):
    b, pos = s["seq_of_token"].long(), s["positions"].long()
    j = torch.arange(s["max_len"], device="cuda")
    seen = j[None] <= pos[:, None]                                   # [T, n]
    at = _slots(s, b[:, None], torch.where(seen, j[None], 0))
    rows = s["rows"].view(-1, s["rows"].shape[2])[at]                # [T, n, width]
    x = _dequantise(rows, s["pool_scale"][at]) if s["fp8"] else rows.float()
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float()
    score = torch.matmul(q, x.transpose(1, 2)) * s["scale"]          # [T, H, n]
    score = score.masked_fill(~seen[:, None], -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    out = torch.matmul(e, x[..., :L]) / e.sum(-1, keepdim=True)
    return out.to(torch.bfloat16)


def _prefill_plain(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    T, H, B = s["q"].shape[0], s["q"].shape[1], cu_q.numel() - 1
    i = torch.arange(s["max_q"], device="cuda")
    j = torch.arange(s["max_k"], device="cuda")
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    iq = (cu_q[:-1, None] + i).clamp_max(T - 1)
    jk = (cu_k[:-1, None] + j).clamp_max(s["v"].shape[0] - 1)
    q = s["q"][iq].float().transpose(1, 2)                           # [B, H, nq, DN + DR]
    rope = s["k_rope"][jk].float()[:, :, None].expand(-1, -1, H, -1)
    k = torch.cat([s["k_nope"][jk].float(), rope], -1).transpose(1, 2)
    v = s["v"][jk].float().transpose(1, 2)
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]          # [B, H, nq, nk]
    seen = (j <= i[:, None] + (nk - nq)[:, None, None]) & (j < nk[:, None, None])
    score.masked_fill_(~seen[:, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    out = torch.matmul(score, v) / score.sum(-1, keepdim=True).clamp_min(1e-30)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu_q[1:].contiguous(), t, right=True).clamp_max(B - 1)
    return out.transpose(1, 2)[b, t - cu_q[b]].to(torch.bfloat16)


def run(s):
    op, fp8 = s["op"], s["fp8"]
    if not own:
        if op == "prefill":
            return _prefill_plain(s)
        if op == "decode":
            return _decode_plain(s)
        if op == "read":
            return _read_plain(s)
        _write_plain(s)
    else:
        import sparse_paged_attention_gb300 as spa
        if op == "prefill":
            return spa.sparse_attn_latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"],
                                                  s["cu_k"], scale=s["scale"])
        pool = spa.LatentPool(s["rows"], s["block_table"], R, s["pool_scale"] if fp8 else None)
        if op == "decode":
            f = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
            return f(s["q_latent"], s["q_rope"], pool, s["positions"], scale=s["scale"],
                     seq_of_token=s["seq_of_token"])
        if op == "read":
            f = spa.sparse_attn_latent_read_fp8 if fp8 else spa.sparse_attn_latent_read
            return f(s["positions"], pool, seq_of_token=s["seq_of_token"])
        f = spa.sparse_attn_latent_write_fp8 if fp8 else spa.sparse_attn_latent_write
        f(s["latent"], s["rope"], s["positions"], pool, seq_of_token=s["seq_of_token"])
    if fp8:
        return {"rows": s["rows"].view(torch.float8_e4m3fn), "scale": s["pool_scale"]}
    return {"rows": s["rows"]}


def work(case):
    op = case["op"]
    if op == "prefill":
        nq = _lengths(case).astype(np.int64)
        nk, H = nq + case["prefix"], case["heads"]
        seen = float((nq * case["prefix"] + nq * (nq + 1) // 2).sum())
        T, S = float(nq.sum()), float(nk.sum())
        return {"bytes": 2.0 * (T * H * (DN + DR + DV) + S * (H * (DN + DV) + DR)),
                "flops": 2.0 * H * (DN + DR + DV) * seen}
    row = L + 2 * R + 4 if case["fp8"] else 2 * (L + R)
    if op == "decode":
        lens = _lengths(case).astype(np.int64)
        n, H = case["q"], case["heads"]
        seen = float(sum(np.maximum(lens - k, 1).sum() for k in range(n)))
        T = case["seqs"] * n
        return {"bytes": float(lens.sum()) * row + 2.0 * T * H * (2 * L + R) + 8.0 * T,
                "flops": 2.0 * H * (2 * L + R) * seen}
    return {"bytes": case["tokens"] * (row + 2.0 * (L + R) + 8), "flops": 0.0}


def _values64(s):
    """The cache's rows in 64 bits, [rows, L + R]."""
    rows = s["rows"].reshape(-1, s["rows"].shape[2])
    if not s["fp8"]:
        return rows.double()
    v = rows.view(torch.float8_e4m3fn).double()
    v[:, L:L + R] += v[:, L + R:]
    return v[:, :L + R] * s["pool_scale"].double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        out = torch.zeros((s["q"].shape[0], case["heads"], DV), dtype=torch.float64, device="cuda")
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["seqs"]):
            n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            rope = s["k_rope"][ck[b]:ck[b + 1]].double()
            hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1)
            for h in range(case["heads"]):
                q = s["q"][cq[b]:cq[b + 1], h].double()
                k = s["k_nope"][ck[b]:ck[b + 1], h].double()
                z = (q[:, :DN] @ k.T + q[:, DN:] @ rope.T) * s["scale"]
                p = torch.softmax(z.masked_fill_(hidden, -math.inf), dim=-1)
                out[cq[b]:cq[b + 1], h] = p @ s["v"][ck[b]:ck[b + 1], h].double()
        return out
    page = case["page"]
    table = s["block_table"].tolist()
    if case["op"] == "decode":
        rows = _values64(s)
        outs = []
        for t, (b, pos) in enumerate(zip(s["seq_of_token"].tolist(), s["positions"].tolist())):
            at = torch.tensor([table[b][p] for p in range(pos // page + 1)], device="cuda") * page
            x = rows[(at[:, None] + torch.arange(page, device="cuda")).reshape(-1)[:pos + 1]]
            z = s["q_latent"][t].double() @ x[:, :L].T + s["q_rope"][t].double() @ x[:, L:].T
            outs.append(torch.softmax(z * s["scale"], dim=-1) @ x[:, :L])
        return torch.stack(outs)
    at = torch.tensor([table[b][x // page] * page + x % page
                       for b, x in zip(s["seq_of_token"].tolist(), s["positions"].tolist())],
                      device="cuda")
    if case["op"] == "read":
        return _values64(s)[at]
    new = torch.cat([s["latent"], s["rope"]], 1).double()
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
