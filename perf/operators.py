"""The operators that serve a batch of requests over a paged cache held in 4 bits, as cases to
measure: each operator in a plain torch form (32-bit arithmetic, rounded once) and as the calls a
user makes of the library.

  tables   page tables, slot map and packed offsets of one step, from the requests' lengths
  store    K/V rows of a step quantised to 4 bits at their slots, and read back
  load     cached rows read back as bf16 (a stored chunk handed to the blend)
  decode   one new token per request attending over its pages
  prompt   causal attention of whole prompts (or chunks), packed one after the other

The 4-bit cache is uint8 [n_pages, hkv, page_size / 16 * 18 D]: for every 16 tokens of a page and
kv head one record of 18 D bytes. A value is scale * code, code in -7 .. 7 (stored + 8 in a nibble),
one bf16 scale per 32 dims: scale = bf16(max|x| / 7), code = round-half-even(x / scale).
  bytes [0, 8 D)       K: [token 16][c 4][group D/32][4], dims 32 group + 8 c + e; byte 2 odd + quad
                       holds e = 4 quad + odd (low nibble) and 4 quad + 2 + odd (high)
  bytes [8 D, 16 D)    V: [half 2][r 8][c 4][group D/32][odd 2][2], token 8 half + 2 c + odd,
                       dims 32 group + 4 r + i, byte i / 2, low nibble first
  bytes [16 D, 18 D)   scales: [token 16][K, V][group D/32] bf16
"""

import math
import random

import numpy as np
import torch

own = False

# (query heads, kv heads, head_dim): the workloads' and the decode tests' head layouts
HEADS = [(4, 2, 64), (32, 8, 128), (64, 8, 128), (16, 16, 128), (32, 16, 64), (16, 1, 64), (32, 2, 128)]
MAX_PROMPT_SCORES = 16 * 32 * 2048 * 2048  # padded score entries of the largest prompt case


def listed():
    return [
        # one decode step of 64 running requests: a page is taken only where one fills up
        {"name": "tables_decode64", "op": "tables", "n_seqs": 64, "max_ctx": 8448, "max_new": 1, "page": 64, "pad": 0,
         "mix": 1},
        # a prefill step of 512 queued prompts, rows padded to a captured graph's size
        {"name": "tables_prefill512", "op": "tables", "n_seqs": 512, "max_ctx": 0, "max_new": 2048, "page": 16,
         "pad": 777, "mix": 2},
        # the K/V rows of a decode step of 64 requests
        {"name": "store_decode64", "op": "store", "n": 64, "hq": 64, "hkv": 8, "d": 128, "page": 64},
        # the rows of the 16 chunks of the long-context request
        {"name": "store_chunks32k", "op": "store", "n": 32768, "hq": 32, "hkv": 8, "d": 128, "page": 64},
        # one 512-token chunk read back for the blend, from a pool of small pages
        {"name": "load_chunk512", "op": "load", "n": 512, "hq": 32, "hkv": 8, "d": 128, "page": 16},
        # the 16 stored chunks of the long-context request read back
        {"name": "load_chunks32k", "op": "load", "n": 32768, "hq": 32, "hkv": 8, "d": 128, "page": 128},
        # a few short chats on a small model
        {"name": "decode_tiny4", "op": "decode", "n_seqs": 4, "max_len": 545, "hq": 4, "hkv": 2, "d": 64, "page": 16,
         "mix": 3},
        # the first token after the long-context request
        {"name": "decode_long32k", "op": "decode", "n_seqs": 1, "max_len": 32897, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "mix": 0},
        # 64 running requests of every length up to the 70B-shaped request's
        {"name": "decode_batch64", "op": "decode", "n_seqs": 64, "max_len": 8449, "hq": 64, "hkv": 8, "d": 128,
         "page": 32, "mix": 4},
        # three short chunks on a small model
        {"name": "prompt_tiny3", "op": "prompt", "n_seqs": 3, "max_len": 256, "hq": 4, "hkv": 2, "d": 64, "pad": 0,
         "mix": 5},
        # queued prompts of every length, packed, with rows of padding behind the last
        {"name": "prompt_ragged40", "op": "prompt", "n_seqs": 40, "max_len": 1087, "hq": 64, "hkv": 8, "d": 128,
         "pad": 45, "mix": 6},
        # the 16 chunks of the long-context request, encoded each on its own
        {"name": "prompt_chunks16x2048", "op": "prompt", "n_seqs": 16, "max_len": 2048, "hq": 32, "hkv": 8, "d": 128,
         "pad": 0, "mix": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "store", "load", "decode", "decode", "prompt", "prompt"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    hq, hkv, d = rng.choice(HEADS)
    mix = rng.randrange(1, 1 << 20)
    if op == "tables":
        prefill = rng.random() < 0.5
        return {"op": op, "n_seqs": _log(rng, 1, 600), "max_ctx": rng.choice([0, _log(rng, 1, 9000)]),
                "max_new": _log(rng, 2, 2048) if prefill else 1, "page": page, "pad": rng.choice([0, _log(rng, 1, 900)]),
                "mix": mix}
    if op in ("store", "load"):
        return {"op": op, "n": _log(rng, 1, 32768 * 1024 // max(1024, hkv * d)), "hq": hq, "hkv": hkv, "d": d,
                "page": page}
    if op == "decode":
        n_seqs = _log(rng, 1, 100)
        most = min(40000, 64 * 8449 * 1024 // (n_seqs * hkv * d) // 2)
        return {"op": op, "n_seqs": n_seqs, "max_len": _log(rng, 1, most), "hq": hq, "hkv": hkv, "d": d, "page": page,
                "mix": rng.choice([0, mix])}
    n_seqs = _log(rng, 1, 64)
    most = min(8192, int(math.sqrt(MAX_PROMPT_SCORES / (n_seqs * hq))))
    return {"op": op, "n_seqs": n_seqs, "max_len": _log(rng, 1, most), "hq": hq, "hkv": hkv, "d": d,
            "pad": rng.choice([0, rng.randrange(1, 100)]), "mix": rng.choice([0, mix])}


def lengths(n, most, mix, least=0):
    """n request lengths up to `most`: all of them `most` where mix is 0, else spread over the range
    with one at `most` (and one at `least`, where there are more than two)."""
    if not mix:
        return [most] * n
    r = random.Random(mix)
    got = [r.randint(min(least + 1, most), most) for _ in range(n)]
    got[r.randrange(n)] = most
    if n > 2:
        got[r.randrange(n)] = least
    return got


def _lens(case):
    """The lengths that a case stands for: (cached, new) of its requests."""
    n = case["n_seqs"]
    if case["op"] == "tables":
        ctx = lengths(n, case["max_ctx"], case["mix"])
        new = lengths(n, case["max_new"], case["mix"] + 1 if case["max_new"] > 1 else 0)
        return ctx, new
    if case["op"] == "decode":
        return [0] * n, lengths(n, case["max_len"], case["mix"])
    return [0] * n, lengths(n, case["max_len"], case["mix"], 1 if case["max_len"] > 1 else 0)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _rows(g, n, h, d, scale=1.0):
    return (scale * torch.randn((n, h, d), generator=g, device="cuda")).bfloat16()


def _page_bytes(page, d):
    return page // 16 * 18 * d


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    op, page = case["op"], case.get("page", 16)
    if op == "tables":
        hq, hkv, d = 4, 2, 64
        ctx, new = _lens(case)
        have = [-(-c // page) for c in ctx]
        need = [-(-(c + w) // page) - h for c, w, h in zip(ctx, new, have)]
        ids = torch.randperm(sum(have) + sum(need) + 9, generator=g, device="cuda").int()
        width = max(h + w for h, w in zip(have, need)) + 1
        table = torch.full((len(ctx), width), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(width, device="cuda") < _ints(have)[:, None]
        table[held] = ids[:sum(have)]
        rows = sum(new) + case["pad"]
        s |= {"ctx": _ints(ctx), "new": _ints(new), "free": ids[sum(have):].contiguous(), "table": table,
              "from": _ints([3])}
        s |= {k: torch.zeros(n, dtype=torch.int32, device="cuda")
              for k, n in (("cu", len(ctx) + 1), ("kv_lens", len(ctx)), ("pos", rows), ("slots", rows), ("to", 1))}
    else:
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        ctx, new = _lens(case) if op in ("decode", "prompt") else ([0], [case["n"]])
        total = sum(new)
        # keys with a channel offset, as cached keys have; values of unit size
        k = _rows(g, total, hkv, d) + 0.5 * _rows(g, 1, hkv, d)
        v = _rows(g, total, hkv, d)
    if op in ("store", "load", "decode"):
        pages = [-(-n // page) for n in new]
        n_pages = sum(pages) + 3
        cache = torch.randint(0, 256, (n_pages, hkv, _page_bytes(page, d)), dtype=torch.uint8, device="cuda",
                              generator=g)  # slots that nothing was stored to hold any bytes
        table = torch.full((len(new), max(max(pages), 1)), -1, dtype=torch.int32, device="cuda")
        ids = torch.randperm(n_pages, generator=g, device="cuda").int()
        table[torch.arange(table.shape[1], device="cuda") < _ints(pages)[:, None]] = ids[:sum(pages)]
        if op == "store" and total <= 256:  # a decode step: one slot in each of many pages
            n_pages = total + 3
            cache = torch.randint(0, 256, (n_pages, hkv, _page_bytes(page, d)), dtype=torch.uint8, device="cuda",
                                  generator=g)
            slots = (torch.randperm(n_pages, generator=g, device="cuda")[:total] * page
                     + torch.randint(0, page, (total,), generator=g, device="cuda")).int()
        else:
            seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), _ints(new), output_size=total)
            starts = _ints([sum(new[:i]) for i in range(len(new))])
            pos = torch.arange(total, device="cuda") - starts[seq]
            slots = (table[seq, pos // page].long() * page + pos % page).int()
        s |= {"cache": cache, "slots": slots}
        if op == "store":
            s |= {"k": k, "v": v}
        else:
            _plain_store(k, v, slots, cache, page)
        if op == "decode":
            s |= {"q": _rows(g, len(new), hq, d), "table": table, "kv_lens": _ints(new)}
            s["out"] = torch.zeros_like(s["q"])
        else:
            s |= {"k_out": torch.zeros_like(k), "v_out": torch.zeros_like(v)}
    if op == "prompt":
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        rows = total + case["pad"]
        fill = _rows(g, case["pad"], hkv, d)
        s |= {"q": _rows(g, rows, hq, d), "k": torch.cat([k, fill]), "v": torch.cat([v, fill]), "cu": _ints(cu)}
        s["out"] = torch.zeros_like(s["q"])  # the rows behind the last prompt stay as they are
    if own:
        import rag_kv_cache_gb300 as cb

        s["plan"] = cb.Plan(1, 1, 0, hq, hkv, d, 1e4)
    return s


def run(s):
    case = s["case"]
    if own:
        return _own_run(case["op"], case.get("page", 0), s)
    return {"tables": _plain_tables, "store": _plain_store_run, "load": _plain_load_run, "decode": _plain_decode,
            "prompt": _plain_prompt}[case["op"]](s)


def _own_run(op, page, s):
    import rag_kv_cache_gb300 as cb

    plan = s["plan"]
    if op == "tables":
        cb.cb_page_tables(plan, s["ctx"], s["new"], page, s["free"], s["table"], s["cu"], s["kv_lens"], s["pos"],
                          s["slots"], s["to"], free_from=s["from"])
        return {k: s[k] for k in ("table", "cu", "kv_lens", "pos", "slots", "to")}
    if op == "store":
        cb.cb_kv4_store(plan, s["k"], s["v"], s["slots"], s["cache"], page)
    if op in ("store", "load"):
        cb.cb_kv4_load(plan, s["cache"], page, s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "decode":
        cb.cb_kv4_decode_attention(plan, s["q"], s["cache"], page, s["table"], s["kv_lens"], s["out"])
    else:
        cb.cb_prompt_attention(plan, s["q"], s["k"], s["v"], s["cu"], s["out"])
    return {"out": s["out"]}


# ---- plain forms ----------------------------------------------------------------------------


def _plain_tables(s):
    page, ctx, new, free, table = s["case"]["page"], s["ctx"].long(), s["new"].long(), s["free"], s["table"]
    have = (ctx + page - 1) // page
    need = (ctx + new + page - 1) // page - have
    first = torch.cumsum(need, 0) - need + s["from"].long()
    nth = torch.arange(table.shape[1], device="cuda") - have[:, None]
    taken = free[(first[:, None] + nth).clamp(0, free.numel() - 1)]
    table = torch.where((nth >= 0) & (nth < need[:, None]), taken, table)
    cu = torch.zeros(len(ctx) + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    row = torch.arange(s["slots"].numel(), device="cuda")
    seq = torch.searchsorted(cu[1:], row, right=True)
    there, seq = seq < len(ctx), seq.clamp(max=len(ctx) - 1)
    pos = torch.where(there, ctx[seq] + row - cu[seq], 0)
    slot = table[seq, pos // page].long() * page + pos % page
    out = {"table": table, "cu": cu, "kv_lens": ctx + new, "pos": pos, "slots": torch.where(there, slot, -1),
           "to": s["from"] + need.sum()}
    return {k: v.int() for k, v in out.items()}


def _quantise(x):
    """Codes (int32, -7 .. 7) [n, h, D] and scales (bf16) [n, h, D / 32]."""
    x = x.float().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    scale = torch.where(x.isfinite().all(-1), top / 7, math.nan).bfloat16()
    step = scale.float()[..., None]
    code = torch.where(step > 0, torch.round(x / step), 0.0).clamp(-7, 7)
    return code.int().flatten(-2), scale


def _record_at(slots, hkv, d, page):
    """Byte offset of each row's record in the cache, [n, hkv], and each row's place in it, [n]."""
    slots = slots.long()
    block = slots // page * hkv * (page // 16) + slots % page // 16
    head = torch.arange(hkv, device="cuda") * (page // 16)
    return (block[:, None] + head) * (18 * d), slots % 16


def _byte_index(slots, hkv, d, page):
    """Offsets in the cache's bytes of the rows' K bytes [n, hkv, 4, D/32, 4], V bytes
    [n, hkv, 8, D/32, 2] and scale bytes [n, hkv, 2, D/32, 2]."""
    at, t = _record_at(slots, hkv, d, page)
    span = lambda n: torch.arange(n, device="cuda")  # noqa: E731
    t, ng = t[:, None], d // 32
    k = (at + t * (d // 2))[..., None] + span(d // 2)
    v = at + 8 * d + (t // 8) * (4 * d) + (t % 8 // 2) * (4 * ng) + (t % 2) * 2
    v = v[..., None, None, None] + span(8)[:, None, None] * (16 * ng) + span(ng)[:, None] * 4 + span(2)
    sc = (at + 16 * d + t * (4 * ng))[..., None] + span(4 * ng)
    return k, v, sc


def _plain_store(k, v, slots, cache, page):
    n, hkv, d = k.shape
    ki, vi, si = _byte_index(slots, hkv, d, page)
    flat = cache.view(-1)
    kc, ks = _quantise(k)
    vc, vs = _quantise(v)
    # K: dims (group, c, quad, nibble, odd) -> bytes (c, group, odd, quad), the nibble inside
    kn = (kc + 8).view(n, hkv, -1, 4, 2, 2, 2).permute(0, 1, 3, 2, 6, 4, 5)
    flat[ki.view(-1)] = (kn[..., 0] + 16 * kn[..., 1]).to(torch.uint8).reshape(-1)
    # V: dims (group, r, byte, nibble) -> bytes (r, group, byte)
    vn = (vc + 8).view(n, hkv, -1, 8, 2, 2).permute(0, 1, 3, 2, 4, 5)
    flat[vi.view(-1)] = (vn[..., 0] + 16 * vn[..., 1]).to(torch.uint8).reshape(-1)
    flat[si.view(-1)] = torch.stack([ks, vs], 2).contiguous().view(torch.uint8).reshape(-1)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).float() - 8


def _values(kb, vb, sb, d):
    """The rows that K bytes [.., D/2], V bytes [.., 8, D/32, 2] and scale bytes [.., 8 D/64] stand for."""
    ng, lead = d // 32, kb.shape[:-1]
    sc = sb.contiguous().view(torch.bfloat16).float().view(*lead, 2, ng, 1)
    n = len(lead)
    keep = tuple(range(n))
    kn = _nibbles(kb.view(*lead, 4, ng, 2, 2)).permute(*keep, n + 1, n, n + 3, n + 4, n + 2)
    vn = _nibbles(vb).permute(*keep, n + 1, n, n + 2, n + 3)
    k = kn.reshape(*lead, ng, 32) * sc[..., 0, :, :]
    v = vn.reshape(*lead, ng, 32) * sc[..., 1, :, :]
    return k.flatten(-2), v.flatten(-2)


def _plain_load(cache, slots, hkv, d, page):
    ki, vi, si = _byte_index(slots, hkv, d, page)
    flat = cache.view(-1)
    return _values(flat[ki], flat[vi], flat[si], d)


def _plain_load_run(s):
    c = s["case"]
    k, v = _plain_load(s["cache"], s["slots"], c["hkv"], c["d"], c["page"])
    return {"k": k.bfloat16(), "v": v.bfloat16()}


def _plain_store_run(s):
    _plain_store(s["k"], s["v"], s["slots"], s["cache"], s["case"]["page"])
    return _plain_load_run(s)


def _softmax(x):
    top = x.amax(-1, keepdim=True)
    x = torch.exp_(x.sub_(top))
    return x.div_(x.sum(-1, keepdim=True))


def _plain_decode(s):
    c, q = s["case"], s["q"].float()
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    n, ng = len(q), d // 32
    rec = s["cache"][s["table"].clamp(min=0).long()]  # [n, pages, hkv, bytes]
    rec = rec.view(n, -1, hkv, page // 16, 18 * d).transpose(1, 2).reshape(n, hkv, -1, 18 * d)
    kb = rec[..., :8 * d].reshape(n, hkv, -1, d // 2)
    vb = rec[..., 8 * d:16 * d].reshape(n, hkv, -1, 2, 8, 4, ng, 2, 2)
    vb = vb.permute(0, 1, 2, 3, 5, 7, 4, 6, 8).reshape(n, hkv, -1, 8, ng, 2)
    k, v = _values(kb, vb, rec[..., 16 * d:].reshape(n, hkv, -1, 4 * ng), d)
    there = torch.arange(k.shape[2], device="cuda") < s["kv_lens"][:, None]  # [n, keys]
    k, v = (torch.where(there[:, None, :, None], x, 0.0) for x in (k, v))
    score = q.view(n, hkv, hq // hkv, d) @ k.transpose(-1, -2) / math.sqrt(d)
    score = score.masked_fill(~there[:, None, None, :], -1e30)  # finite: a request without keys gives zeros
    return {"out": (_softmax(score) @ v).reshape(n, hq, d).bfloat16()}


def _plain_prompt(s):
    c, cu = s["case"], s["cu"].long()
    hq, hkv, d, n, most = c["hq"], c["hkv"], c["d"], c["n_seqs"], c["max_len"]
    at = torch.arange(most, device="cuda")
    rows = (cu[:-1, None] + at).clamp(max=len(s["q"]) - 1)
    q = s["q"][rows].float().view(n, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    k, v = (s[x][rows].float().transpose(1, 2) for x in ("k", "v"))
    score = (q @ k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(n, hkv, -1, most, most)
    score.masked_fill_(at > at[:, None], -math.inf)
    o = (_softmax(score).view(n, hkv, -1, most) @ v).view(n, hkv, -1, most, d).permute(0, 3, 1, 2, 4)
    row = torch.arange(len(s["q"]), device="cuda")
    seq = torch.searchsorted(cu[1:], row, right=True)
    there, seq = seq < n, seq.clamp(max=n - 1)
    o = o.reshape(n, most, hq, d)[seq, (row - cu[seq]).clamp(0, most - 1)]
    return {"out": torch.where(there[:, None, None], o.bfloat16(), s["out"])}


# ---- what a pass cannot do without ------------------------------------------------------------


def work(case):
    op, page = case["op"], case.get("page", 16)
    if op == "tables":
        ctx, new = _lens(case)
        have = [-(-c // page) for c in ctx]
        need = sum(-(-(c + w) // page) - h for c, w, h in zip(ctx, new, have))
        rows = sum(new) + case["pad"]
        # lengths in; free pages in, table entries out; offsets, lengths, positions and slots out
        return {"bytes": 4 * (2 * len(ctx) + 2 * need + 2 * len(ctx) + 1 + 2 * rows + 2), "flops": 2 * rows}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    held = hkv * 18 * d // 16  # bytes of a cached token
    if op in ("store", "load"):
        n = case["n"]
        both = n * hkv * d * 4
        return {"bytes": (2 if op == "store" else 1) * (both + n * held) + 4 * n, "flops": 4 * n * hkv * d}
    lens = _lens(case)[1]
    if op == "decode":
        pages = sum(-(-n // page) for n in lens)
        return {"bytes": sum(lens) * held + 4 * len(lens) * hq * d + 4 * pages + 4 * len(lens),
                "flops": 4 * hq * d * sum(lens)}
    return {"bytes": sum(lens) * d * (4 * hq + 4 * hkv) + 4 * len(lens),
            "flops": 4 * hq * d * sum(n * (n + 1) // 2 for n in lens)}


# ---- the same from the definitions, in 64 bits -------------------------------------------------


def _exact_quantised(x):
    """scale * code of every 32 dims, in 64 bits."""
    x = x.double()
    out = torch.empty_like(x)
    for g in range(x.shape[-1] // 32):
        part = x[..., 32 * g:32 * g + 32]
        scale = (part.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double()
        out[..., 32 * g:32 * g + 32] = scale * torch.round(part / scale.clamp(min=1e-300))
    return out


def _exact_rows(cache, slots, d, page):
    """The values at `slots`, read nibble by nibble as the record's layout says: K, V [n, hkv, D]."""
    pages = (slots // page).long()
    blk, t = (slots % page // 16).long(), (slots % 16).long()
    hkv = cache.shape[1]
    rec = cache.view(cache.shape[0], hkv, page // 16, 18 * d)[pages, :, blk]  # [n, hkv, 18 D]
    pick = lambda off: torch.gather(rec, 2, off[:, None, None].expand(-1, hkv, 1))[..., 0].int()  # noqa: E731
    k = torch.empty((len(slots), hkv, d), dtype=torch.float64, device=cache.device)
    v = torch.empty_like(k)
    ng = d // 32
    for dim in range(d):
        g, e = dim // 32, dim % 32
        word = t * (d // 2) + (e // 8 * ng + g) * 4
        byte = pick(word + e % 2 * 2 + e % 8 // 4)
        kcode = (byte >> (4 * (e % 4 // 2))) % 16 - 8
        word = 8 * d + t // 8 * (4 * d) + e // 4 * (16 * ng) + t % 8 // 2 * (4 * ng) + 4 * g + t % 2 * 2
        byte = pick(word + e % 4 // 2)
        vcode = (byte >> (4 * (e % 2))) % 16 - 8
        for which, code, to in ((0, kcode, k), (1, vcode, v)):
            off = 16 * d + t * (4 * ng) + which * 2 * ng + 2 * g
            bits = (pick(off) + 256 * pick(off + 1)) << 16
            to[..., dim] = code.double() * bits.view(torch.float32).double()
    return k, v


def _exact_attention(q, k, v, visible):
    """q [m, hq, D] over k, v [keys, hkv, D]: row i sees the keys below visible[i]."""
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    out = torch.empty_like(q, dtype=torch.float64)
    hidden = torch.arange(len(k), device=q.device) >= visible[:, None]
    for h in range(hq):
        a = q[:, h].double() @ k[:, h * hkv // hq].double().T / math.sqrt(d)
        out[:, h] = torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ v[:, h * hkv // hq].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case.get("page", 16)
    if op == "tables":
        ctx, new = _lens(case)
        free, table, at = s["free"].tolist(), s["table"].tolist(), 3
        rows = s["slots"].numel()
        cu, pos, slots = [0], [0] * rows, [-1] * rows
        for i, (c, w) in enumerate(zip(ctx, new)):
            for p in range(-(-c // page), -(-(c + w) // page)):
                table[i][p] = free[at]
                at += 1
            for j in range(w):
                pos[cu[-1] + j] = c + j
                slots[cu[-1] + j] = table[i][(c + j) // page] * page + (c + j) % page
            cu.append(cu[-1] + w)
        got = {"table": table, "cu": cu, "kv_lens": [c + w for c, w in zip(ctx, new)], "pos": pos, "slots": slots,
               "to": [at]}
        return {k: np.array(v, dtype=np.int32) for k, v in got.items()}
    if op == "store":
        return {"k": _exact_quantised(s["k"]), "v": _exact_quantised(s["v"])}
    if op == "load":
        k, v = _exact_rows(s["cache"], s["slots"], case["d"], page)
        return {"k": k, "v": v}
    lens = _lens(case)[1]
    out = s["out"].double()
    at = 0
    for i, n in enumerate(lens):
        if op == "decode" and n:
            tok = torch.arange(n, device="cuda")
            k, v = _exact_rows(s["cache"], s["table"][i][tok // page].long() * page + tok % page, case["d"], page)
            out[i] = _exact_attention(s["q"][i:i + 1], k, v, _ints([n]))[0]
        elif op == "prompt":
            rows = slice(at, at + n)
            out[rows] = _exact_attention(s["q"][rows], s["k"][rows], s["v"][rows],
                                         torch.arange(1, n + 1, device="cuda"))
        at += n
    return {"out": out}
