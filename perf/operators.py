"""Decoding from a paged K/V cache and evicting from it: the measured cases and their plain forms.

Three kinds of call over one cache layout ([slots, 64, Hkv, d] pages, a block table per
sequence, lengths on the device):

  decode   attention of the newest q_len tokens of every sequence over its cached keys,
           optionally with a prefix that all sequences share and that is stored once,
           optionally adding each key's softmax weight to a running total per kv-head;
  evict    keep the first `sink`, the last `recent` and the heaviest other tokens of every
           (sequence, kv-head), `budget` in all, and move their rows to fresh pages.

With `own` false, `run` computes them with elementary torch operations in 32 bits; with
`own` true it calls the library.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 64
GOLDEN = 0.6180339887498949


def _lens(case):
    """Cached tokens of every sequence: max_len for the first, the others spread over
    1..max_len (ragged) or all equal."""
    B, n = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [n] * B
    return [n if b == 0 else 1 + int(((b * GOLDEN) % 1.0) * n * 0.999) for b in range(B)]


def _pages(n):
    return -(-n // PAGE)


def listed():
    layer = {"q_heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16", "q_len": 1, "ragged": False, "prefix": 0, "weights": False}

    def dec(name, **kw):
        return {"name": name, "op": "decode", **layer, **kw}

    def evi(name, **kw):
        return {"name": name, "op": "evict", "q_heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16", "ragged": False, **kw}

    return [
        # the smallest call: one short sequence of the two-head test problem, where latency is all
        dec("decode_b1_1k_d64", batch=1, max_len=1024, q_heads=2, kv_heads=2, dim=64),
        # one user with a full 128K context, FP8 cache: few rows, a long axis to split
        dec("decode_b1_128k_fp8", batch=1, max_len=131072, dtype="fp8_e4m3"),
        # the step after the paged prefill batch: four sequences up to 128K, very unequal
        dec("decode_b4_ragged_128k", batch=4, max_len=131072, ragged=True),
        # a serving batch checking four drafted tokens a sequence
        dec("decode_b48_q4_ragged_4k", batch=48, max_len=4096, q_len=4, ragged=True),
        # a few chats behind one system prompt
        dec("prefix_b8_4k", batch=8, max_len=256, ragged=True, prefix=4000),
        # a batch of questions about one long document
        dec("prefix_b64_32k", batch=64, max_len=1024, ragged=True, prefix=32768),
        # a wide sampling batch over one document, FP8 cache
        dec("prefix_b128_16k_fp8", batch=128, max_len=512, ragged=True, prefix=16384, dtype="fp8_e4m3"),
        # decoding while the weights that eviction goes by are collected
        dec("weights_b4_32k", batch=4, max_len=32768, weights=True),
        dec("weights_b32_ragged_8k_fp8", batch=32, max_len=8192, ragged=True, dtype="fp8_e4m3", weights=True),
        # a small cache cut to a quarter
        evi("evict_b1_1k_d64", batch=1, max_len=1024, q_heads=2, kv_heads=2, dim=64, budget=256, sink=4, recent=64),
        # four 32K caches cut to the 25 % budget
        evi("evict_b4_32k", batch=4, max_len=32768, budget=8192, sink=64, recent=1024),
        # a ragged FP8 serving batch; the shorter sequences lose nothing
        evi("evict_b32_ragged_64k_fp8", batch=32, max_len=65536, ragged=True, dtype="fp8_e4m3", budget=8192, sink=4, recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("decode", "prefix", "weights", "evict"))
    fp8 = rng.random() < 0.4
    dim = 128 if fp8 or rng.random() < 0.75 else 64
    kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8))
    if rng.random() < 0.3:
        kv_heads, group = 8, 4
    case = {"op": "evict" if kind == "evict" else "decode", "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
            "dtype": "fp8_e4m3" if fp8 else "bf16", "batch": _log(rng, 1, 128 if kind == "prefix" else 64), "ragged": rng.random() < 0.7}
    if kind == "evict":
        n = min(_log(rng, 2, 131072), 6_000_000 // (case["batch"] * kv_heads))
        budget = max(1, min(int(n * rng.uniform(0.05, 0.9)), 900_000 // (case["batch"] * kv_heads)))
        sink = rng.randint(0, min(8, budget // 2))
        case |= {"max_len": n, "budget": budget, "sink": sink, "recent": rng.randint(0, (budget - sink) // 2)}
        return case
    q_len = rng.choice((1, 1, 1, 2, 3, 4, 8))
    rows = case["batch"] * case["q_heads"] * q_len
    most = min(131072, 900_000 // (case["batch"] * kv_heads) * 2, 24_000_000 // rows)
    n = _log(rng, 1, max(1, min(most, 2048) if kind == "prefix" else most))
    prefix = _log(rng, 1, max(1, min(32768, 48_000_000 // rows))) if kind == "prefix" else 0
    case |= {"max_len": n, "q_len": q_len, "prefix": prefix, "weights": kind == "weights"}
    return case


def _codes(x):
    """e4m3 codes and the per-tensor scale of a bf16 tensor."""
    scale = max(float(x.abs().max()), 1e-6) / 448.0
    scale = float(torch.tensor(scale, dtype=torch.float32))
    return (x / scale).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, Hq, Hkv, d = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    fp8 = case["dtype"] == "fp8_e4m3"

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    lens = _lens(case)
    prefix = case.get("prefix", 0)
    need, pre = [_pages(n) for n in lens], _pages(prefix)
    slots = sum(need) + pre
    perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    starts = torch.tensor([pre + sum(need[:b]) for b in range(B)], device="cuda")
    col = torch.arange(max(need), device="cuda")
    # entries past a sequence's pages point at its last page, as unused entries of a table do
    at = starts[:, None] + torch.minimum(col[None, :], torch.tensor(need, device="cuda")[:, None] - 1)
    table = perm[at].contiguous()
    k = normal(slots, PAGE, Hkv, d)
    v = normal(slots, PAGE, Hkv, d)
    # the first tokens of a sequence draw much of the attention
    first = perm[:1] if prefix else table[:, 0].contiguous()
    direction = normal(Hkv, d)
    k[first.long(), :4] += 0.25 * direction
    s = {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "table": table, "case": dict(case), "k_scale": 1.0, "v_scale": 1.0, "q_scale": 1.0}
    if fp8:
        k, s["k_scale"] = _codes(k)
        v, s["v_scale"] = _codes(v)
    s["k"], s["v"] = k, v
    if case["op"] == "decode":
        T = B * case["q_len"]
        q = normal(T, Hq, d) + 0.25 * direction.repeat_interleave(Hq // Hkv, 0)
        if fp8:
            q, s["q_scale"] = _codes(q)
        s |= {"q": q, "out": torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda"), "lse": torch.zeros((Hq, T), device="cuda")}
        s["prefix_table"] = perm[:pre].contiguous() if prefix else None
        if case["weights"]:
            shape = (B, Hkv, max(need) * PAGE)
            s["w_in"] = torch.rand(shape, generator=g, device="cuda") ** 4
            s["w_out"] = torch.zeros(shape, device="cuda")
        if own:
            from block_sparse_attention_oam_b200 import stem as S
            s["S"] = S
            s["plan"] = S.Decode(B, Hq, Hkv, d, max_kv_len=case["max_len"], q_len=case["q_len"], dtype=case["dtype"], q_scale=s["q_scale"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], prefix_len=prefix, weights=case["weights"])
            s["cache"] = S.PagedKV(k, v, table)
            s["ws"] = S.decode_workspace(s["plan"])
        return s
    # running totals of softmax weights: a heavy tail, and keys that nothing has looked at
    shape = (B, Hkv, max(need) * PAGE)
    w = torch.rand(shape, generator=g, device="cuda") ** 8
    s["w"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.1, torch.zeros((), device="cuda"), w)
    fresh = _pages(case["budget"])
    s["new_table"] = torch.randperm(B * fresh, generator=g, device="cuda").to(torch.int32).view(B, fresh)
    s["new_k"] = torch.zeros((B * fresh, PAGE, Hkv, d), dtype=k.dtype, device="cuda")
    s["new_v"] = torch.zeros_like(s["new_k"])
    s["new_w"] = torch.zeros((B, Hkv, fresh * PAGE), device="cuda")
    s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["kept"] = torch.zeros((B, Hkv, case["budget"]), dtype=torch.int32, device="cuda")
    if own:
        from block_sparse_attention_oam_b200 import stem as S
        s["S"] = S
        s["plan"] = S.Evict(B, Hkv, d, max_kv_len=case["max_len"], budget=case["budget"], sink=case["sink"], recent=case["recent"], dtype=case["dtype"])
        s["cache"] = S.PagedKV(k, v, table)
        s["fresh"] = S.PagedKV(s["new_k"], s["new_v"], s["new_table"])
        s["ws"] = S.evict_workspace(s["plan"])
    return s


def run(s):
    case = s["case"]
    if case["op"] == "decode":
        if own:
            s["S"].stem_decode(s["plan"], s["q"], s["cache"], s["lens"], prefix_table=s["prefix_table"], weights_in=s.get("w_in"), weights_out=s.get("w_out"),
                               out=s["out"], lse=s["lse"], ws=s["ws"])
            got = {"out": s["out"], "lse": s["lse"]}
            return got | {"weights": s["w_out"]} if case["weights"] else got
        return _decode_plain(s)
    if own:
        s["S"].stem_evict(s["plan"], s["cache"], s["lens"], s["w"], s["fresh"], kv_lens_out=s["new_lens"], weights_out=s["new_w"], keep=s["kept"], ws=s["ws"])
        return {"kept": s["kept"], "lens": s["new_lens"], "k": s["new_k"], "v": s["new_v"], "weights": s["new_w"]}
    return _evict_plain(s)


def _decode_plain(s):
    case = s["case"]
    B, n, Hq, Hkv, d = case["batch"], case["q_len"], case["q_heads"], case["kv_heads"], case["dim"]
    G = Hq // Hkv
    q = (s["q"].float() * s["q_scale"]).view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d) * (1.0 / math.sqrt(d))
    k = s["k"][s["table"].long()].float().mul_(s["k_scale"]).view(B, -1, Hkv, d).permute(0, 2, 3, 1)
    scores = torch.matmul(q, k)                                              # [B, Hkv, n * G, L]
    del k
    L = scores.shape[-1]
    pos = torch.arange(L, device=q.device)
    limit = s["lens"][:, None].long() - n + 1 + torch.arange(n, device=q.device)[None, :]           # keys of row t
    seen = pos[None, None, :] < limit[:, :, None]                                                   # [B, n, L]
    scores = torch.where(seen[:, None, :, None, :], scores.view(B, Hkv, n, G, L), -math.inf).view(B, Hkv, n * G, L)
    top = scores.amax(-1)
    if case["prefix"]:
        P = case["prefix"]
        at = s["prefix_table"].long()
        kp = s["k"][at].float().mul_(s["k_scale"]).view(-1, Hkv, d)[:P].permute(1, 2, 0)            # [Hkv, d, P]
        flat = q.permute(1, 0, 2, 3).reshape(Hkv, B * n * G, d)
        ps = torch.matmul(flat, kp).view(Hkv, B, n * G, P)
        top = torch.maximum(top, ps.amax(-1).permute(1, 0, 2))
    base = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    scores = torch.exp(scores - base[..., None])
    total = scores.sum(-1)
    v = s["v"][s["table"].long()].float().mul_(s["v_scale"]).view(B, -1, Hkv, d).permute(0, 2, 1, 3)
    o = torch.matmul(scores, v)
    del v
    if case["prefix"]:
        ps = torch.exp(ps - base.permute(1, 0, 2)[..., None])
        vp = s["v"][at].float().mul_(s["v_scale"]).view(-1, Hkv, d)[:P].permute(1, 0, 2)
        o = o + torch.matmul(ps.view(Hkv, B * n * G, P), vp).view(Hkv, B, n * G, d).permute(1, 0, 2, 3)
        total = total + ps.sum(-1).permute(1, 0, 2)
        del ps
    none = total == 0
    o = torch.where(none[..., None], torch.zeros_like(o), o / total[..., None])
    lse = torch.log(total) + base
    out = o.view(B, Hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(B * n, Hq, d).to(torch.bfloat16)
    got = {"out": out, "lse": lse.view(B, Hkv, n, G).permute(1, 3, 0, 2).reshape(Hq, B * n)}
    if case["weights"]:
        w = torch.where(none[..., None], torch.zeros_like(scores), scores / total[..., None]).sum(2)
        held = pos[None, None, :] < s["lens"][:, None, None]
        got["weights"] = torch.where(held, s["w_in"][..., :L] + w, s["w_out"])
    return got


def _evict_plain(s):
    case = s["case"]
    B, Hkv, d, budget = case["batch"], case["kv_heads"], case["dim"], case["budget"]
    w, lens = s["w"], s["lens"].long()[:, None, None]
    L = w.shape[-1]
    pos = torch.arange(L, device=w.device)[None, None, :]
    held = pos < lens
    forced = (pos < case["sink"]) | (pos >= lens - case["recent"])
    # three classes, each by weight, each by index: sorted by weight first, then stably by class
    rank = torch.where(torch.isnan(w), -math.inf, w)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kind = torch.where(held, torch.where(forced, 0, 1), 2).expand(B, Hkv, L)
    order = order.gather(-1, torch.sort(kind.gather(-1, order), dim=-1, stable=True).indices)
    take = order[..., :budget]
    many = torch.minimum(lens, torch.full_like(lens, budget))
    place = torch.arange(take.shape[-1], device=w.device)[None, None, :]
    take = torch.sort(torch.where(place < many, take, L), dim=-1).values     # kept positions, ascending
    live = (place < many).expand(B, Hkv, -1)
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=w.device)
    kept[..., :take.shape[-1]] = torch.where(live, take, -1).to(torch.int32)
    b, h, i = live.nonzero(as_tuple=True)
    j = take[b, h, i]
    old, new = s["table"][b, j // PAGE].long(), s["new_table"][b, i // PAGE].long()
    nk, nv, nw = torch.zeros_like(s["new_k"]), torch.zeros_like(s["new_v"]), torch.zeros_like(s["new_w"])
    kind = torch.uint8 if case["dtype"] == "fp8_e4m3" else s["k"].dtype      # moves bytes: indexing takes no 8-bit floats
    nk.view(kind)[new, i % PAGE, h] = s["k"].view(kind)[old, j % PAGE, h]
    nv.view(kind)[new, i % PAGE, h] = s["v"].view(kind)[old, j % PAGE, h]
    nw[b, h, i] = w[b, h, j]
    return {"kept": kept, "lens": many.view(B).to(torch.int32), "k": nk, "v": nv, "weights": nw}


def work(case):
    lens, Hkv, d = _lens(case), case["kv_heads"], case["dim"]
    es = 1 if case["dtype"] == "fp8_e4m3" else 2
    row = Hkv * d * es
    if case["op"] == "evict":
        moved = sum(min(n, case["budget"]) for n in lens)
        # every weight is read where something is to be chosen; kept rows, indices and weights are written
        read = sum(n * Hkv * 4 for n in lens)
        return {"bytes": read + moved * (4 * row + Hkv * 8), "flops": 0}
    rows = case["q_len"] * case["q_heads"]
    total = sum(lens) + case["prefix"]
    size = total * 2 * row + len(lens) * rows * (d * (es + 2) + 4)
    if case["weights"]:
        size += sum(lens) * Hkv * 8
    seen = sum(lens) + len(lens) * case["prefix"]
    return {"bytes": size, "flops": 4 * rows * seen * d}


def exact(case, seed):
    """The definition in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    with torch.no_grad():
        return (_exact_decode if case["op"] == "decode" else _exact_evict)(case, s)


def _rows64(cache, pages, n, scale):
    """The first n tokens of a page list, as doubles [Hkv, n, d]."""
    slots = [int(p) for p in pages.tolist()][:_pages(n)]
    parts = [cache[p] for p in slots]
    flat = torch.cat(parts, 0)[:n] if parts else cache[0][:0]
    return (flat.to(torch.float64) * scale).transpose(0, 1).contiguous()


def _exact_decode(case, s):
    n, Hq, Hkv, d = case["q_len"], case["q_heads"], case["kv_heads"], case["dim"]
    G, sigma = Hq // Hkv, case["dim"] ** -0.5
    out, lse, weights = [], [], []
    if case["prefix"]:
        pk = _rows64(s["k"], s["prefix_table"], case["prefix"], s["k_scale"])
        pv = _rows64(s["v"], s["prefix_table"], case["prefix"], s["v_scale"])
    for b, length in enumerate(_lens(case)):
        k = _rows64(s["k"], s["table"][b], length, s["k_scale"])
        v = _rows64(s["v"], s["table"][b], length, s["v_scale"])
        extra = 0
        if case["prefix"]:
            k, v, extra = torch.cat([pk, k], 1), torch.cat([pv, v], 1), case["prefix"]
        w = torch.zeros((Hkv, length), dtype=torch.float64, device=k.device)
        for t in range(n):
            q = (s["q"][b * n + t].to(torch.float64) * s["q_scale"]).view(Hkv, G, d)
            see = max(0, length - n + t + 1) + extra
            if see == 0:
                out.append(torch.zeros((Hq, d), dtype=torch.float64, device=k.device))
                lse.append(torch.full((Hq,), -math.inf, dtype=torch.float64, device=k.device))
                continue
            logits = sigma * torch.einsum("hgd,hjd->hgj", q, k[:, :see])
            z = torch.logsumexp(logits, -1)
            p = torch.exp(logits - z[..., None])
            out.append(torch.einsum("hgj,hjd->hgd", p, v[:, :see]).reshape(Hq, d))
            lse.append(z.reshape(Hq))
            w[:, :see - extra] += p[..., extra:].sum(1)
        if case["weights"]:
            total = torch.zeros(s["w_out"].shape[1:], dtype=torch.float64, device=k.device)
            total[:, :length] = s["w_in"][b, :, :length].double() + w
            weights.append(total)
    got = {"out": torch.stack(out), "lse": torch.stack(lse, 1)}
    return got | {"weights": torch.stack(weights)} if case["weights"] else got


def _exact_evict(case, s):
    import numpy as np
    budget, Hkv = case["budget"], case["kv_heads"]
    B = case["batch"]
    w = s["w"].double().cpu().numpy()
    kept = np.full((B, Hkv, budget), -1, dtype=np.int32)
    lens = np.zeros(B, dtype=np.int32)
    weights = np.zeros(tuple(s["new_w"].shape), dtype=np.float64)
    for b, n in enumerate(_lens(case)):
        lens[b] = m = min(n, budget)
        for h in range(Hkv):
            if n <= budget:
                chosen = np.arange(n)
            else:
                ends = np.concatenate([np.arange(case["sink"]), np.arange(n - case["recent"], n)])
                middle = np.arange(case["sink"], n - case["recent"])
                heaviest = middle[np.lexsort((middle, -w[b, h, middle]))][: budget - len(ends)]
                chosen = np.sort(np.concatenate([ends, heaviest]))
            kept[b, h, :m] = chosen
            weights[b, h, :m] = w[b, h, chosen]
    # rows are moved as they are: their values are those of the cache
    spots = torch.from_numpy(kept).cuda().long()
    moved = {}
    for name in ("k", "v"):
        new = torch.zeros(tuple(s["new_" + name].shape), dtype=torch.float64, device="cuda")
        for b in range(B):
            m = int(lens[b])
            src = s[name].view(torch.uint8 if case["dtype"] == "fp8_e4m3" else torch.int16)[s["table"][b].long()].flatten(0, 1)  # [tokens, Hkv, d]
            rows = torch.gather(src, 0, spots[b, :, :m].t()[:, :, None].expand(-1, -1, src.shape[-1])).view(s[name].dtype).double()
            padded = torch.zeros((s["new_table"].shape[1] * PAGE,) + tuple(rows.shape[1:]), dtype=torch.float64, device="cuda")
            padded[:m] = rows
            new[s["new_table"][b].long()] = padded.view(-1, PAGE, *rows.shape[1:])
        moved[name] = new
    return {"kept": torch.from_numpy(kept), "lens": torch.from_numpy(lens), "k": moved["k"], "v": moved["v"], "weights": torch.from_numpy(weights)}
