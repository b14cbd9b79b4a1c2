"""Workloads of the paged-cache operators: rotary positions, appending to a paged
cache, attention of new tokens over it, and copying its pages.

Each operator has a plain form of elementary torch operations (``own`` false) and
the framework's call (``own`` true).  The cache of one layer is three pools:
k and v pages [pages][kv heads][page tokens][head dim] in bf16, and pooled block
keys [pages][kv heads][head dim] in fp32, a block's mean key standing in the slot
of the block's last page.  Token p of sequence b lies in page
``table[b, p // page]`` at offset ``p % page``.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(name, tokens, hq, hkv, d, rot, interleaved, grad, scaling, far):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "grad": grad, "scaling": scaling, "far": far}


def _append(name, seqs, new, ctx, hkv, d, page, block, mix):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "hkv": hkv, "d": d, "page": page,
            "block": block, "mix": mix}


def _attn(name, seqs, new, ctx, hq, hkv, d, page, block, topk, mix):
    return {"name": name, "op": "attn", "seqs": seqs, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "block": block, "topk": topk, "mix": mix}


def _pages(name, pages, moves, layers, hkv, d, page):
    return {"name": name, "op": "pages", "pages": pages, "moves": moves, "layers": layers, "hkv": hkv, "d": d,
            "page": page}


def listed():
    return [
        # a training step's q and k at the 32K shape, whole heads rotated
        _rope("rope_train", 32768, 32, 32, 128, 128, False, False, "none", 32768),
        # its gradient: odd length, grouped heads, half of each head, pairs side by side, far positions
        _rope("rope_grad", 4 * 8191, 24, 8, 128, 64, True, True, "bands", 1 << 20),
        # one new token of each of 64 running sequences
        _append("append_step", 64, 1, 32768, 8, 128, 64, 512, 3),
        # prompts of several requests written in chunks
        _append("append_chunk", 4, 8192, 32768, 8, 128, 64, 512, 7),
        # the smallest call: one token of one short sequence
        _attn("step_smallest", 1, 1, 1000, 8, 2, 64, 16, 64, 4, 0),
        # a decode step with block selection, 8 sequences with 32K caches, a kv head per q head
        _attn("step_select", 8, 1, 32768, 32, 32, 128, 64, 512, 3, 0),
        # a decode step of a full-attention layer, uneven lengths, grouped heads
        _attn("step_full", 16, 1, 49152, 32, 8, 128, 32, 512, 0, 2),
        # the last chunk of a 32K prompt with block selection
        _attn("chunk_select", 1, 4096, 32768, 32, 8, 128, 64, 512, 3, 0),
        # a chunk of a full-attention layer
        _attn("chunk_full", 1, 2048, 32768, 32, 8, 128, 64, 512, 0, 0),
        # several requests' chunks of uneven sizes, five q heads to a kv head, small blocks
        _attn("chunk_uneven", 7, 500, 9000, 20, 4, 64, 32, 128, 6, 5),
        # forked sequences get their own last page, in every layer
        _pages("pages_fork", 200, 16, 8, 8, 128, 64),
        # a pool compacted after many requests have left
        _pages("pages_compact", 8192, 2500, 1, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "pages"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "rope":
        hq, hkv = rng.choice([(hq, hkv), (32, 8), (32, 32)])
        rot = rng.choice([d, d, d // 2, 16])
        most = 32768 * 64 * 128 // ((hq + hkv) * d)
        return {"op": "rope", "tokens": _log(rng, 1, min(most, 100000)), "hq": hq, "hkv": hkv, "d": d, "rot": rot,
                "interleaved": rng.random() < 0.5, "grad": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "bands"]), "far": _log(rng, 1000, 1 << 20)}
    page = rng.choice([16, 32, 64, 128])
    if op == "pages":
        layers = rng.choice([1, 1, 2, 5])
        each = layers * hkv * page * d
        most = min(20000, 8192 * 8 * 64 * 128 // each)
        pages = _log(rng, 40, max(41, most))
        return {"op": "pages", "pages": pages, "moves": _log(rng, 1, max(1, min(3 * pages // 10, 4000))), "layers": layers,
                "hkv": hkv, "d": d, "page": page}
    block = rng.choice([b for b in (64, 128, 256, 512, 1024, 2048) if b >= page])
    if op == "append":
        seqs = _log(rng, 1, 48)
        new = rng.choice([1, 1, _log(rng, 2, 8192)])
        new = max(1, min(new, 32768 // seqs))
        ctx = max(new, _log(rng, max(64, new), max(64, min(65536, (1 << 20) // seqs))))
        return {"op": "append", "seqs": seqs, "new": new, "ctx": ctx, "hkv": hkv, "d": d, "page": page, "block": block,
                "mix": rng.randrange(1, 1000)}
    seqs = _log(rng, 1, 32)
    new = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 64, 4096)])
    topk = rng.choice([0, 1, 2, 3, 3, 4, 8, 12])
    cells = (1 << (32 if topk else 30)) // (hq * seqs)
    new = max(1, min(new, cells // 2048))
    most = min(65536, cells // new, (1 << 30) // (seqs * hkv * d))
    ctx = _log(rng, max(64, min(new, most)), max(64, most))
    return {"op": "attn", "seqs": seqs, "new": min(new, ctx), "ctx": ctx, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "block": block, "topk": topk, "mix": rng.randrange(0, 1000)}


def _lengths(case):
    """(new tokens, cache length with them) of each sequence: even for mix 0, else spread below the first one's."""
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    if case["mix"] == 0:
        return [new] * n, [ctx] * n
    r = random.Random(case["mix"])
    nq, lens = [new], [ctx]
    for _ in range(n - 1):
        length = r.randint(max(1, ctx // 8), ctx)
        lens.append(length)
        nq.append(0 if new > 1 and r.random() < 0.1 else min(length, r.randint((new + 7) // 8, new)))
    return nq, lens


def _frequencies(rot, scaling):
    """Radians a position for each pair, in 64 bits: base 10000, plain, interpolated by 8, or the slow
    pairs interpolated by 8 and the fast ones kept, with a ramp over the turns in 8192 positions."""
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        f = f / 8
    elif scaling == "bands":
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / 8 * (1 - keep)
    return f


def _magnitude(case):
    return 0.1 * math.log(8) + 1 if case.get("scaling") == "bands" else 1.0


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.bfloat16)


def _cache(case, g, nq, lens):
    """Pools with shuffled pages, the page table (-1 where a sequence has no page) and the lengths."""
    page, hkv, d, block = case["page"], case["hkv"], case["d"], case["block"]
    dev = g.device
    counts = [-(-x // page) for x in lens]
    width = -(-max(lens) // block) * (block // page)
    total = sum(counts)
    pages = total + 5
    order = torch.randperm(pages, generator=g, device=dev)[:total]
    seq = torch.from_numpy(np.repeat(np.arange(len(lens)), counts)).to(dev)
    col = torch.from_numpy(np.concatenate([np.arange(c) for c in counts])).to(dev)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    table[seq, col] = order.to(torch.int32)
    k, v = _normal(g, pages, hkv, page, d), _normal(g, pages, hkv, page, d)
    # keys of a block share an offset, so that the pooled keys tell blocks apart
    blocks = sum(-(-x // block) for x in lens)
    first = np.concatenate([[0], np.cumsum([-(-x // block) for x in lens])[:-1]])
    of_page = torch.from_numpy(np.concatenate([f + np.arange(c) * page // block for f, c in zip(first, counts)])).to(dev)
    offset = 0.5 * _normal(g, blocks, hkv, d)
    k[order] = k[order] + offset[of_page][:, :, None, :]
    # pooled keys of the complete blocks
    kbar = torch.zeros(pages, hkv, d, device=dev)
    per = block // page
    full = [x // block * per for x in lens]
    if sum(full):
        of = torch.cat([table[b, :f] for b, f in enumerate(full)]).long()
        kbar[of[per - 1::per]] = (k[of].sum(2, dtype=torch.float64).view(-1, per, hkv, d).sum(1) / block).float()
    cu = np.concatenate([[0], np.cumsum(nq)])
    return {"k_pages": k, "v_pages": v, "kbar_pages": kbar, "table": table, "cu_host": cu, "lens_host": np.array(lens),
            "cu": torch.from_numpy(cu).to(dev, torch.int32), "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(seed)
    dev = g.device
    s = {"case": case}
    if case["op"] == "rope":
        t = case["tokens"]
        s["q"], s["k"] = _normal(g, t, case["hq"], case["d"]), _normal(g, t, case["hkv"], case["d"])
        first = torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=dev)
        s["positions"] = ((torch.arange(t, device=dev) + first) % case["far"]).to(torch.int32)
        s["freqs"] = torch.from_numpy(_frequencies(case["rot"], case["scaling"])).to(dev)
    elif case["op"] == "pages":
        shape = (case["layers"], case["pages"], case["hkv"])
        s["k_pages"], s["v_pages"] = (_normal(g, *shape, case["page"], case["d"]) for _ in range(2))
        s["kbar_pages"] = torch.randn(*shape, case["d"], generator=g, device=dev)
        at = torch.randperm(case["pages"], generator=g, device=dev).to(torch.int32)
        s["src"], s["dst"] = at[:case["moves"]].contiguous(), at[case["moves"]:2 * case["moves"]].contiguous()
    else:
        nq, lens = _lengths(case)
        s.update(_cache(case, g, nq, lens))
        if case["op"] == "append":
            s["k"], s["v"] = (_normal(g, sum(nq), case["hkv"], case["d"]) for _ in range(2))
        else:
            s["q"] = _normal(g, sum(nq), case["hq"], case["d"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _turn(x, positions, freqs, interleaved, grad, magnitude):
    """Rotated x [T][H][D] in 32 bits, angles in 64."""
    angle = positions.double()[:, None] * freqs
    c, s = (angle.cos() * magnitude).float()[:, None], (angle.sin() * magnitude).float()[:, None]
    s = -s if grad else s
    rot = 2 * freqs.numel()
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.stack((a * c - b * s, b * c + a * s), -1) if interleaved else torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y.flatten(-2) if interleaved else y, x[..., rot:]), -1)


def _rows(s):
    """The sequence and position of each new token."""
    t = torch.arange(int(s["cu_host"][-1]), device=s["cu"].device)
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    return b, t - s["cu"][b] + (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[b]


def _plain_rope(s):
    c = s["case"]
    return {n: _turn(s[n], s["positions"], s["freqs"], c["interleaved"], c["grad"], _magnitude(c)).bfloat16() for n in ("q", "k")}


def _plain_append(s):
    c = s["case"]
    page, block = c["page"], c["block"]
    b, pos = _rows(s)
    to, off = s["table"][b, pos // page].long(), pos % page
    s["k_pages"][to, :, off] = s["k"]
    s["v_pages"][to, :, off] = s["v"]
    # the blocks that this call completes
    lens, nq = s["lens_host"], np.diff(s["cu_host"])
    before, after = (lens - nq) // block, lens // block
    done = after - before
    if done.sum():
        per = block // page
        seq = np.repeat(np.arange(len(lens)), done)
        col = np.repeat(before, done) + np.arange(done.sum()) - np.repeat(np.cumsum(done) - done, done)
        cols = torch.from_numpy(col[:, None] * per + np.arange(per)).to(b.device)
        of = s["table"][torch.from_numpy(seq).to(b.device)[:, None], cols].long()
        s["kbar_pages"][of[:, -1]] = (s["k_pages"][of].sum((1, 3), dtype=torch.float64) / block).float()
    return {n: s[n] for n in ("k_pages", "v_pages", "kbar_pages")}


def _plain_attn(s):
    c = s["case"]
    page, block, hkv, d, topk = c["page"], c["block"], c["hkv"], c["d"], c["topk"]
    group = c["hq"] // hkv
    table = s["table"].clamp(min=0).long()
    seqs, length, new = table.shape[0], int(s["lens_host"].max()), int(np.diff(s["cu_host"]).max())
    b, pos = _rows(s)
    j = torch.arange(b.numel(), device=b.device) - s["cu"][b]
    x = s["q"].new_zeros(seqs, new, hkv, group, d)
    x[b, j] = s["q"].view(-1, hkv, group, d)
    x = x.permute(0, 2, 3, 1, 4)  # [seq][kv head][group][new][d]
    k, v = (p[table].transpose(1, 2).reshape(seqs, hkv, -1, d)[:, :, :length].float() for p in (s["k_pages"], s["v_pages"]))
    first = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None]
    # positions [seq][1][1][new][1]; a shorter chunk's rows behind its end stand at the last key
    at = (first + torch.arange(new, device=b.device)).clamp(max=length - 1)[:, None, None, :, None]
    key = torch.arange(length, device=b.device)
    hidden = key > at
    idx = None
    if topk:
        n = -(-length // block)
        past = s["kbar_pages"][table[:, block // page - 1::block // page][:, :n]].transpose(1, 2).double()  # [seq][kv head][n][d]
        score = torch.matmul(x.double(), past[:, :, None].transpose(-1, -2))
        blocks = torch.arange(n, device=b.device)
        mine = (at // block).expand(score.shape[:-1] + (1,))
        score.masked_fill_(blocks >= mine, -math.inf)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :topk - 1]
        best = torch.where(best < mine, best, n)
        taken = torch.zeros(score.shape[:-1] + (n + 1,), dtype=torch.bool, device=b.device)
        taken.scatter_(-1, torch.cat((best, mine), -1), True)
        hidden = hidden | ~taken[..., key // block]
        idx = torch.full(score.shape[:-1] + (topk,), n, device=b.device)
        idx[..., :best.shape[-1]] = best
        idx[..., -1:] = mine
        idx = torch.sort(idx, -1).values
        idx = torch.where(idx < n, idx, -1).to(torch.int32)
        idx = idx.permute(0, 3, 1, 2, 4)[b, j].reshape(-1, c["hq"], topk)
    w = torch.matmul(x.float() / math.sqrt(d), k[:, :, None].transpose(-1, -2))
    w.masked_fill_(hidden, -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, v[:, :, None]) / total
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2)[b, j].reshape(-1, c["hq"])
    out = out.permute(0, 3, 1, 2, 4)[b, j].reshape(-1, c["hq"], d).bfloat16()
    return {"out": out, "lse": lse} if idx is None else {"out": out, "lse": lse, "idx": idx}


def _plain_pages(s):
    src, dst = s["src"].long(), s["dst"].long()
    names = ("k_pages", "v_pages", "kbar_pages")
    return {n: s[n].index_copy_(1, dst, s[n].index_select(1, src)) for n in names}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_rope(s):
    from long_context_sparse_moba_gb300 import ops
    c = s["case"]
    call = ops.rope_bwd if c["grad"] else ops.rope
    q, k = call(s["q"], s["k"], s["positions"], s["freqs"], interleaved=c["interleaved"], magnitude=_magnitude(c))
    return {"q": q, "k": k}


def _own_append(s):
    from long_context_sparse_moba_gb300 import ops
    c = s["case"]
    ops.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["kbar_pages"], s["table"], s["cu"], s["lens"], c["new"],
                     c["block"])
    return {n: s[n] for n in ("k_pages", "v_pages", "kbar_pages")}


def _own_attn(s):
    from long_context_sparse_moba_gb300 import ops
    c = s["case"]
    every = s["table"].shape[1] * c["page"] // c["block"]
    out, lse, idx = ops.paged_attn(s["q"], s["k_pages"], s["v_pages"], s["kbar_pages"], s["table"], s["cu"], s["lens"],
                                   c["new"], c["block"], c["topk"] or every, with_idx=c["topk"] > 0)
    return {"out": out, "lse": lse} if idx is None else {"out": out, "lse": lse, "idx": idx}


def _own_pages(s):
    from long_context_sparse_moba_gb300 import ops
    ops.page_copy(s["k_pages"], s["v_pages"], s["kbar_pages"], s["src"], s["dst"])
    return {n: s[n] for n in ("k_pages", "v_pages", "kbar_pages")}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn": _own_attn, "pages": _own_pages}[op](s)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "pages": _plain_pages}[op](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        values = case["tokens"] * (case["hq"] + hkv) * d
        return {"bytes": 4 * values + 4 * case["tokens"], "flops": 3 * values * case["rot"] / d}
    if case["op"] == "pages":
        one = case["layers"] * hkv * d * (4 * case["page"] + 4)
        return {"bytes": 2 * case["moves"] * one + 8 * case["moves"], "flops": 0}
    nq, lens = _lengths(case)
    block, page = case["block"], case["page"]
    nbytes = flops = 0.0
    if case["op"] == "append":
        for n, length in zip(nq, lens):
            nbytes += 8 * n * d * hkv + 4 * n / page
            done = length // block - (length - n) // block
            if done:  # keys of the first completed block that were there before, and the pooled keys
                nbytes += hkv * d * (2 * ((length - n) % block) + 4 * done)
                flops += hkv * d * done * block
        return {"bytes": nbytes, "flops": flops}
    group = case["hq"] // hkv
    for n, length in zip(nq, lens):
        if not n:
            continue
        pos = np.arange(length - n, length, dtype=np.float64)
        mine = pos // block
        if case["topk"]:
            picks = np.minimum(case["topk"] - 1, mine)
            keys = pos % block + 1 + picks * block
            past = mine[-1]
            # blocks that some row picks, were the picks even: every row is one draw of its picks
            share = np.minimum(1.0, picks / np.maximum(mine, 1))
            read = past * (1 - float(np.prod((1 - share) ** group)))
            own_first = mine[0]
            read = max(read, past - own_first) * block + length - past * block
            nbytes += hkv * past * d * 4 + n * case["hq"] * case["topk"] * 4
            flops += 2.0 * d * group * hkv * float(mine.sum())
        else:
            keys, read = pos + 1, length
        nbytes += 4.0 * read * hkv * d + n * case["hq"] * (4 * d + 4)
        flops += 4.0 * d * case["hq"] * float(keys.sum())
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(x, positions, freqs, interleaved, grad, magnitude):
    """The pairs as complex numbers, multiplied by magnitude * exp(+-i angle)."""
    pairs = freqs.numel()
    y = x.double().clone()
    place = torch.arange(pairs, device=x.device)
    re, im = (2 * place, 2 * place + 1) if interleaved else (place, place + pairs)
    angle = torch.outer(positions.double(), freqs) * (-1.0 if grad else 1.0)
    z = torch.complex(y[..., re], y[..., im]) * torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_append(s):
    page, block = s["case"]["page"], s["case"]["block"]
    kp, vp, kb = s["k_pages"].double(), s["v_pages"].double(), s["kbar_pages"].double()
    table = s["table"].long()
    for b, (lo, hi, length) in enumerate(zip(s["cu_host"][:-1], s["cu_host"][1:], s["lens_host"])):
        lo, hi, length = int(lo), int(hi), int(length)
        p = torch.arange(length - (hi - lo), length, device=kp.device)
        kp[table[b, p // page], :, p % page] = s["k"][lo:hi].double()
        vp[table[b, p // page], :, p % page] = s["v"][lo:hi].double()
        for blk in range((length - (hi - lo)) // block, length // block):
            of = table[b, blk * block // page:(blk + 1) * block // page]
            kb[of[-1]] = kp[of].mean((0, 2))
    return {"k_pages": kp, "v_pages": vp, "kbar_pages": kb}


def _exact_attn(s):
    c = s["case"]
    page, block, hkv, d, topk = c["page"], c["block"], c["hkv"], c["d"], c["topk"]
    group = c["hq"] // hkv
    q = s["q"].double().view(-1, hkv, group, d)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device)
    for b, (lo, hi, length) in enumerate(zip(s["cu_host"][:-1], s["cu_host"][1:], s["lens_host"])):
        lo, hi, length = int(lo), int(hi), int(length)
        of = s["table"][b, :-(-length // page)].long()
        step = max(1, (1 << 27) // (length * group))
        for h in range(hkv):
            keys = s["k_pages"][of, h].reshape(-1, d)[:length].double()
            values = s["v_pages"][of, h].reshape(-1, d)[:length].double()
            means = s["kbar_pages"][of[block // page - 1::block // page], h].double()
            for t in range(lo, hi, step):
                x = q[t:min(hi, t + step), h]
                at = (torch.arange(t, t + x.shape[0], device=q.device) + length - hi)[:, None, None]
                seen = (torch.arange(length, device=q.device) <= at).expand(-1, group, -1)
                if topk:
                    number = torch.arange(means.shape[0], device=q.device)
                    left = (x @ means.T).masked_fill(number >= at // block, -math.inf)
                    open_ = (torch.arange(length, device=q.device) // block == at // block).expand(-1, group, -1).clone()
                    for _ in range(min(topk - 1, means.shape[0])):
                        most = left.amax(-1, keepdim=True)
                        pick = torch.where(left == most, number, means.shape[0]).amin(-1, keepdim=True)
                        open_ |= (torch.arange(length, device=q.device) // block == pick) & (most > -math.inf)
                        left = left.masked_fill(number == pick, -math.inf)
                    seen = seen & open_
                logit = (x @ keys.T * d ** -0.5).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(logit, -1)
                lse[t:t + x.shape[0], h] = z
                out[t:t + x.shape[0], h] = torch.exp(logit - z[..., None]) @ values
    got = {"out": out.view(-1, c["hq"], d), "lse": lse.view(-1, c["hq"])}
    return {**got, "idx": None} if topk else got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {n: _exact_turn(s[n], s["positions"], s["freqs"], case["interleaved"], case["grad"], _magnitude(case)) for n in ("q", "k")}
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    src, dst = s["src"].tolist(), s["dst"].tolist()
    got = {n: s[n].double() for n in ("k_pages", "v_pages", "kbar_pages")}
    for n in got:
        for layer in range(case["layers"]):
            got[n][layer][dst] = got[n][layer][src]
    return got
