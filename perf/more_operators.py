"""Measured cases of several continuations of one prompt in the 8-bit paged cache: decode attention of requests that share a
prefix, the choice of the next beams over beams and vocabulary, and the reordering of the beams' states.

Each case runs in a plain form (elementary torch operations, float32 or float64) or, where ``own`` is true, through the
library's entry points on the same buffers.

The 8-bit cache: a page holds P tokens of every kv head; the block of a (layer, page, kv head) is

    K codes [P][d] | V codes [P][d] | K scale f32, V scale f32, 8 zero bytes | K lo [d] | K hi [d] | zeros to a multiple of 128 bytes

with one byte per code (INT8: code + 128; E4M3: the number's pattern).  Token rows are d bytes; the 16-byte chunks of each
128-byte line of a code section lie in an order of their own (``chunk_order``).  Tokens of the page that is not complete yet
are BF16 rows of the tail slab [layer][request slot][kv head][K|V][P][d].

Shared prefix: the requests of a batch lie group by group; the first ``shared`` pages of a group's requests are the same pages.
Beams: candidate (beam, token) has score[beam] + log softmax(logits[beam])[token]; the largest come first, the lowest
(beam, token) first among equal ones.
Reordering: beam j of an item continues parents[j].  The first child of a beam keeps its request slot; the others take the
slots of beams without a child, both in ascending order, and the beam's tail rows are copied there.
"""
import math
import weakref

import numpy as np
import torch

own = False

TOP = {"int8": 127.0, "e4m3": 448.0}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------- cases
def _shared(name, **kw):
    return dict(dict(op="shared", layout=1, pad=0.0), name=name, **kw)


def _beam(name, **kw):
    return dict(dict(op="beam", first=False, done=0.0, masked=0.0, gap=0), name=name, **kw)


def _reorder(name, **kw):
    return dict(dict(op="reorder", layout=1, dead=0.0), name=name, **kw)


def listed():
    return [
        # two samples of a short prompt in float32 at the smallest geometry: latency
        _shared("shared_pair_f32", groups=1, size_lo=2, size_hi=2, q_heads=4, kv_heads=2, d=64, page=16, fmt="int8", dtype="f32",
                out="f32", shared_lo=320, shared_hi=320, own_lo=3, own_hi=25),
        # four prompts of 8K tokens with four beams each, a little way into their answers
        _shared("shared_4x4_8k", groups=4, size_lo=4, size_hi=4, q_heads=32, kv_heads=8, d=128, page=64, fmt="e4m3", dtype="bf16",
                out="bf16", shared_lo=6000, shared_hi=8192, own_lo=1, own_hi=300),
        # eight beams of one very long document
        _shared("shared_8_131k", groups=1, size_lo=8, size_hi=8, q_heads=32, kv_heads=8, d=128, page=64, fmt="int8", dtype="bf16",
                out="bf16", shared_lo=130048, shared_hi=130048, own_lo=100, own_hi=1000),
        # 64 samples of one 32K prompt, 64 query heads
        _shared("shared_64_32k", groups=1, size_lo=64, size_hi=64, q_heads=64, kv_heads=8, d=128, page=64, fmt="e4m3",
                dtype="bf16", out="bf16", shared_lo=32768, shared_hi=32768, own_lo=64, own_hi=1024),
        # conversations behind system prompts: groups of any size, single requests among them, some places of the batch empty
        _shared("shared_ragged", groups=12, size_lo=1, size_hi=9, q_heads=32, kv_heads=4, d=64, page=32, fmt="int8", dtype="f32",
                out="f32", shared_lo=500, shared_hi=6000, own_lo=0, own_hi=2500, pad=0.1),
        # one prompt, two beams, a small vocabulary, the first step: latency
        _beam("beam_2_997", batch=1, beams=2, vocab=997, n_out=2, dtype="f32", first=True),
        # eight prompts with four beams, twice as many candidates as beams
        _beam("beam_8x4_32k", batch=8, beams=4, vocab=32768, n_out=8, dtype="bf16"),
        # an odd vocabulary in float32 with finished beams and a grammar's mask
        _beam("beam_6x5_50021", batch=6, beams=5, vocab=50021, n_out=10, dtype="f32", done=0.2, masked=0.9),
        # a full batch over a large vocabulary
        _beam("beam_32x8_131k", batch=32, beams=8, vocab=131072, n_out=16, dtype="bf16"),
        # two layers at the smallest geometry: latency
        _reorder("reorder_2_layers", layers=2, batch=1, beams=3, q_heads=4, kv_heads=2, d=64, page=16, fmt="int8", n_lo=333,
                 n_hi=333),
        # 36 layers, four prompts with four beams
        _reorder("reorder_4x4", layers=36, batch=4, beams=4, q_heads=32, kv_heads=8, d=128, page=64, fmt="e4m3", n_lo=4000,
                 n_hi=5029),
        # 36 layers, sixteen prompts with eight beams, some of them out of candidates
        _reorder("reorder_16x8", layers=36, batch=16, beams=8, q_heads=32, kv_heads=8, d=128, page=64, fmt="int8", n_lo=7000,
                 n_hi=20000, dead=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "beam", "beam", "reorder"])
    layout = rng.randrange(1 << 20)
    if op == "beam":
        batch, beams = _log(rng, 1, 32), _log(rng, 1, 16)
        vocab = _log(rng, 30, min(131072, (1 << 25) // (batch * beams)))
        c = _beam("", batch=batch, beams=beams, vocab=vocab, n_out=min(rng.choice([1, beams, 2 * beams]), beams * vocab),
                  dtype=rng.choice(["f32", "bf16"]), first=rng.random() < 0.2, done=rng.choice([0.0, 0.0, 0.3]),
                  masked=rng.choice([0.0, 0.0, 0.5, 0.99]), gap=rng.choice([0, 0, 8, 13]))
    else:
        kv = rng.choice([1, 2, 4, 8])
        geom = dict(q_heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv, d=rng.choice([64, 128, 128]),
                    page=rng.choice([16, 32, 64, 64]), fmt=rng.choice(["int8", "e4m3"]), layout=layout)
        if op == "shared":
            groups = _log(rng, 1, 16)
            size = _log(rng, 1, 64 // groups)
            hi = _log(rng, geom["page"], min(131072, (1 << 20) // (groups * size), (1 << 18) // groups))
            own_hi = _log(rng, 1, 2000)
            c = _shared("", groups=groups, size_lo=rng.choice([1, size]), size_hi=size, shared_lo=hi // rng.choice([1, 2, 30]),
                        shared_hi=hi, own_lo=own_hi // rng.choice([1, 3, 40]), own_hi=own_hi, dtype=rng.choice(["f32", "bf16"]),
                        out=rng.choice(["f32", "bf16"]), pad=rng.choice([0.0, 0.0, 0.2]), **geom)
        else:
            n = _log(rng, 1, 20000)
            c = _reorder("", layers=rng.randint(1, 36), batch=_log(rng, 1, 16), beams=_log(rng, 2, 8), n_lo=n // rng.choice([1, 2, 9]),
                         n_hi=n, dead=rng.choice([0.0, 0.0, 0.2]), **geom)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------- geometry
def _sections(case):
    """Byte offsets inside a block: (V codes, scales, lo, hi), and the block's size."""
    P, d = case["page"], case["d"]
    s = 2 * P * d
    return P * d, s, s + 16, s + 16 + d, -(-(s + 16 + 2 * d) // 128) * 128


def chunk_order(P, d, is_v):
    """Stored place of every logical 16-byte chunk (row-major: token, then channel) of a code section."""
    c = np.arange(P * d // 16)
    t = c * 16 // d
    turn = 2 * ((t >> 1) & 3) if is_v else (4 * (t & 1) if d == 128 else 0 * t)
    return torch.from_numpy((c & ~7) | ((c & 7) ^ turn)).cuda()


def _grouping(case):
    """(requests of each group, its shared pages, the length of every request)."""
    r, P = np.random.default_rng([case["layout"], 11]), case["page"]
    sizes = r.integers(case["size_lo"], case["size_hi"] + 1, case["groups"])
    shared = r.integers(case["shared_lo"], case["shared_hi"] + 1, case["groups"]) // P
    sizes[0], shared[0] = case["size_hi"], case["shared_hi"] // P
    total = int(sizes.sum())
    more = r.integers(case["own_lo"], case["own_hi"] + 1, total)
    more[0] = case["own_hi"]
    n = np.repeat(shared, sizes) * P + more
    empty = r.random(total) < case["pad"]
    empty[0] = False
    n[empty] = 0
    return sizes, shared, n


def _family(case):
    """(parents [batch][beams], lengths [batch][beams]) of a reordering."""
    r = np.random.default_rng([case["layout"], 13])
    B, K = case["batch"], case["beams"]
    n = np.repeat(r.integers(case["n_lo"], case["n_hi"] + 1, B)[:, None], K, 1)
    luck = r.dirichlet(np.full(K, 1.0), B)
    parents = np.stack([r.choice(K, K, p=luck[b]) for b in range(B)])
    parents[r.random((B, K)) < case["dead"]] = -1
    return parents, n


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _activations(shape, gen, dtype):
    """[..., heads, d] with a deviation of its own for every channel and two loud channels a head."""
    h, d = shape[-2:]
    sigma = torch.exp(0.5 * torch.randn(h, d, generator=gen, device="cuda"))
    loud = torch.rand(h, d, generator=gen, device="cuda").topk(2, dim=1).indices
    sigma.scatter_(1, loud, sigma.gather(1, loud) * 8)
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


# ------------------------------------------------------------------------------------------------- plain forms
def _blocks(k, v, case, orders):
    """k, v: [..., P, d] float32.  The blocks [..., block bytes] as a write leaves them."""
    P, d = case["page"], case["d"]
    ov, os_, ol, oh, size = _sections(case)
    out = torch.zeros(*k.shape[:-2], size, dtype=torch.uint8, device="cuda")
    for x, order, at, sc in ((k, orders[0], 0, 0), (v, orders[1], ov, 4)):
        big = x.abs().amax(dim=(-2, -1))
        y = x * TOP[case["fmt"]] / big[..., None, None]
        if case["fmt"] == "int8":
            val = y.round().clamp(-127, 127)
            kind = lambda t: (t + 128).to(torch.uint8)   # noqa: E731
        else:
            val = y.clamp(-448, 448).to(torch.float8_e4m3fn).float() + 0.0
            kind = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)   # noqa: E731
        rows = torch.empty(*k.shape[:-2], P * d // 16, 16, dtype=torch.uint8, device="cuda")
        rows[..., order, :] = kind(val).reshape(*k.shape[:-2], P * d // 16, 16)
        out[..., at:at + P * d] = rows.reshape(*k.shape[:-2], P * d)
        out[..., os_ + sc:os_ + sc + 4] = (big / TOP[case["fmt"]])[..., None].contiguous().view(torch.uint8)
        if sc == 0:
            out[..., ol:ol + d], out[..., oh:oh + d] = kind(val.amin(dim=-2)), kind(val.amax(dim=-2))
    return out


def _dequantised(blocks, case, orders):
    """blocks: [B, pages, heads, size].  K and V [B, heads, pages * P, d]."""
    P, d = case["page"], case["d"]
    B, n, heads, _ = blocks.shape
    ov, os_, _, _, _ = _sections(case)
    scale = blocks[..., os_:os_ + 8].contiguous().view(torch.float32)
    got = []
    for i, at in enumerate((0, ov)):
        code = blocks[..., at:at + P * d].reshape(B, n, heads, P * d // 16, 16)[:, :, :, orders[i]]
        code = code.float() - 128 if case["fmt"] == "int8" else code.view(torch.float8_e4m3fn).float()
        x = code.reshape(B, n, heads, P, d) * scale[..., i, None, None]
        got.append(x.permute(0, 2, 1, 3, 4).reshape(B, heads, n * P, d))
    return got


def _plain_shared(s):
    """Group by group: scores against the prefix for all of the group's query heads at once, against each request's own pages and
    tail rows, one softmax over both."""
    case, P, d = s["case"], s["case"]["page"], s["case"]["d"]
    heads, G = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    bt, n, slot, out = s["bt"].long(), s["n"].long(), s["slot"].long(), []
    b0 = 0
    for R, pre, most in zip(s["sizes"], s["pre"], s["most"]):
        at = slice(b0, b0 + R)
        b0 += R
        q = s["q"][at].float().reshape(R, heads, G, d).transpose(0, 1)                          # [heads, R, G, d]
        here = n[at] > 0
        left = (n[at] - pre * P).clamp(min=0)                                                   # tokens of its own
        own_p = torch.arange(pre, pre + most, device="cuda")
        there = own_p < (n[at] // P)[:, None]                                                   # [R, most]
        k, v = _dequantised(s["pool"][0][torch.where(there, bt[at, pre:pre + most], 0 * own_p)], case, s["orders"])
        tail = s["tail"][0][slot[at]].float()                                                   # [R, heads, 2, P, d]
        live = torch.arange(P, device="cuda") < (left % P)[:, None]
        tail = torch.where(live[:, None, None, :, None], tail, torch.zeros_like(tail))
        k, v = (torch.cat([a, tail[:, :, i]], 2).transpose(0, 1) for i, a in enumerate((k, v)))  # [heads, R, own, d]
        seen = torch.cat([there.repeat_interleave(P, 1), live], 1)[None, :, None]
        x = (torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)).masked_fill(~seen, -math.inf)   # [heads, R, G, own]
        if pre:
            first = s["first"][b0 - R]                                                          # a request that holds the prefix
            pk, pv = (a[0] for a in _dequantised(s["pool"][0][bt[first, :pre]][None], case, s["orders"]))
            y = torch.matmul(q.reshape(heads, R * G, d), pk.transpose(1, 2)).reshape(heads, R, G, pre * P) / math.sqrt(d)
            y = y.masked_fill(~here[None, :, None, None], -math.inf)
        else:
            y = x[..., :0]
        m = torch.cat([x, y], 3).amax(3, keepdim=True)
        m = torch.where(m.isinf(), torch.zeros_like(m), m)
        p, w = torch.exp(x - m), torch.exp(y - m)
        o = torch.matmul(p, v)
        if pre:
            o = o + torch.matmul(w.reshape(heads, R * G, pre * P), pv).reshape(heads, R, G, d)
        total = p.sum(3, keepdim=True) + w.sum(3, keepdim=True)
        o = o / torch.where(total > 0, total, torch.ones_like(total))
        out.append(o.transpose(0, 1).reshape(R, heads * G, d))
    return torch.cat(out).to(DT[case["out"]])


def _plain_beam(s):
    case = s["case"]
    B, K, V = case["batch"], case["beams"], case["vocab"]
    x = s["logits"].double()
    m = x.amax(2, keepdim=True)
    alive = ~m.isinf()
    x = x - torch.where(alive, m, torch.zeros_like(m))
    key = s["scores"].double()[:, :, None] + (x - torch.log(torch.exp(x).sum(2, keepdim=True)).masked_fill(~alive, 0.0))
    done = s["done"].bool()[:, :, None]
    pad = torch.arange(V, device="cuda") == s["eos"]
    key = torch.where(done, torch.where(pad, s["scores"].double()[:, :, None], torch.full_like(key, -math.inf)), key)
    top, at = torch.sort(key.reshape(B, K * V), dim=1, descending=True, stable=True)
    top, at = top[:, :case["n_out"]], at[:, :case["n_out"]]
    none = top == -math.inf
    at = at.masked_fill(none, -1)
    return {"scores": top.float(), "tokens": torch.where(none, at, at % V).int(), "parents": torch.where(none, at, at // V).int()}


def _plain_reorder(s):
    case, P = s["case"], s["case"]["page"]
    B, K = case["batch"], case["beams"]
    par, slot, n = s["parents"].long(), s["slot"].long().view(B, K), s["n"].long().view(B, K)
    of = par[:, :, None] == torch.arange(K, device="cuda")                                      # [B, child, parent]
    first = (of & (of.long().cumsum(1) == 1)).any(2)
    free = torch.sort(of.any(1).long(), dim=1, stable=True).indices                             # beams without a child come first
    take = torch.gather(free, 1, ((~first).long().cumsum(1) - 1).clamp(min=0))
    some, at = par >= 0, par.clamp(min=0)
    new_slot = torch.gather(slot, 1, torch.where(first, at, take))
    src = torch.where(some & ~first, torch.gather(slot, 1, at), new_slot)
    new_n = torch.where(some, torch.gather(n, 1, at), torch.zeros_like(n))
    rows = (torch.arange(P, device="cuda") < (new_n % P)[:, :, None]).reshape(1, B * K, 1, 1, P, 1)
    dst, src = new_slot.reshape(-1), src.reshape(-1)
    s["tail"][:, dst] = torch.where(rows, s["tail"][:, src], s["tail"][:, dst])
    table = s["bt"].view(B, K, -1)
    table = torch.where(some[:, :, None], torch.gather(table, 1, at[:, :, None].expand_as(table)), torch.full_like(table, -1))
    return {"tail": s["tail"], "table": table.reshape(B * K, -1), "lens": new_n.reshape(-1).int(), "slots": new_slot.reshape(-1).int()}


# ------------------------------------------------------------------------------------------------- prepare
class _Keep:
    pass


def _handle(s, layers, slots, pages, per_req):
    """The context that a program keeps, its 8-bit pool and tail bound to it."""
    import int2_rotated_paged_oscar_gb300 as osc
    c = s["case"]
    cfg = osc.make_config(num_layers=layers, n_q_heads=c.get("q_heads", 1), n_kv_heads=c.get("kv_heads", 1),
                          head_dim=c.get("d", 64), page_size=c.get("page", 16), sink=0, recent=1, max_requests=slots,
                          max_pages_per_req=per_req, num_pages=pages)
    ctx = osc.oscar_create(cfg)
    if "pool" not in s:   # the choice of beams needs a context, not a cache's contents
        s["pool"], s["tail"] = (torch.zeros(f(cfg), dtype=torch.uint8, device="cuda")
                                for f in (osc.oscar_kv8_pool_bytes, osc.oscar_kv8_tail_bytes))
    osc.oscar_kv8_bind(ctx, osc.KV8_INT8 if c.get("fmt") == "int8" else osc.KV8_E4M3, s["pool"], s["tail"])
    s.update(osc=osc, cfg=cfg, ctx=ctx, dt=osc.DTYPE_F32 if c.get("dtype") == "f32" else osc.DTYPE_BF16,
             odt=osc.DTYPE_F32 if c.get("out") == "f32" else osc.DTYPE_BF16)
    s["keep"] = _Keep()
    weakref.finalize(s["keep"], osc.oscar_destroy, ctx)


def _filled_pool(s, pages, gen):
    """A pool of one layer whose pages hold quantised activations, a few thousand blocks at a time."""
    case = s["case"]
    P, d, heads = case["page"], case["d"], case["kv_heads"]
    pool = torch.empty(pages, heads, _sections(case)[-1], dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (heads * P * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        level = torch.exp(0.3 * torch.randn(n, 1, heads, 1, generator=gen, device="cuda"))   # pages differ in loudness
        k, v = (_activations((n, P, heads, d), gen, torch.float32) * level for _ in range(2))
        k += 0.7 * torch.randn(n, 1, heads, d, generator=gen, device="cuda")                 # and in what they are about
        pool[at:at + n] = _blocks(*(x.to(torch.bfloat16).float().permute(0, 2, 1, 3) for x in (k, v)), case, s["orders"])
    return pool[None]


def _slab(case, layers, slots, gen):
    heads, P, d = case["kv_heads"], case["page"], case["d"]
    return _activations((layers * slots, 2 * P, heads, d), gen, torch.bfloat16).view(layers, slots, 2, P, heads, d) \
        .permute(0, 1, 4, 2, 3, 5).contiguous()


def prepare(case, seed):
    gen, rng = _gen(seed), np.random.default_rng([seed, 5])
    s = {"case": case}
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()   # noqa: E731
    if case["op"] == "shared":
        P, d, heads = case["page"], case["d"], case["kv_heads"]
        s["orders"] = (chunk_order(P, d, False), chunk_order(P, d, True))
        sizes, shared, n = _grouping(case)
        B, group = len(n), np.repeat(np.arange(len(sizes)), sizes)
        mine = np.maximum(n // P - shared[group], 0)                    # pages of its own
        mine[n == 0] = 0
        pages = int(shared.sum() + mine.sum()) + 3
        ids, per_req = rng.permutation(pages), int((shared[group] + mine).max()) + 1
        bt, at = np.full((B, per_req), -1, np.int32), int(shared.sum())
        cut = np.concatenate([[0], np.cumsum(shared)])
        for b in range(B):
            if n[b]:
                g = group[b]
                bt[b, :shared[g]] = ids[cut[g]:cut[g + 1]]
                bt[b, shared[g]:shared[g] + mine[b]] = ids[at:at + mine[b]]
                at += mine[b]
        starts = np.concatenate([[0], np.cumsum(sizes)])
        holder = [int(b0 + (n[b0:b1] > 0).argmax()) for b0, b1 in zip(starts[:-1], starts[1:])]
        s.update(sizes=sizes.tolist(), pre=shared.tolist(), most=[int(mine[group == g].max()) for g in range(len(sizes))],
                 first=dict(zip(starts[:-1].tolist(), holder)), bt=dev(bt), n=dev(n), slot=dev(rng.permutation(B + 1)[:B]),
                 starts=dev(starts), shared=dev(shared), most_shared=int(shared.max()), most_own=max(1, int((n - shared[group] * P).max())))
        s["pool"], s["tail"] = _filled_pool(s, pages, gen), _slab(case, 1, B + 1, gen)
        s["q"] = _activations((B, case["q_heads"], d), gen, DT[case["dtype"]]) * 0.7
        s["out"] = torch.empty(B, case["q_heads"], d, dtype=DT[case["out"]], device="cuda")
        if own:
            _handle(s, 1, B + 1, pages, per_req)
            size = s["osc"].oscar_kv8_shared_workspace_size(s["cfg"], B, len(sizes), s["most_shared"], s["most_own"])
            s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    elif case["op"] == "beam":
        B, K, V, N = case["batch"], case["beams"], case["vocab"], case["n_out"]
        wide = torch.empty(B, K, V + case["gap"], dtype=DT[case["dtype"]], device="cuda")
        x = torch.randn(B, K, V, generator=gen, device="cuda") * 2.0 - 2.0 * torch.log1p(torch.arange(V, device="cuda") / 50.0)
        x += torch.randn(B, 1, V, generator=gen, device="cuda") * 2.0          # the beams of an item are of one mind
        if case["masked"]:
            x.masked_fill_(torch.rand(B, K, V, generator=gen, device="cuda") < case["masked"], -math.inf)
        wide[:, :, :V] = x
        scores = -20.0 * torch.rand(B, K, generator=gen, device="cuda")
        if case["first"]:
            scores[:, 0], scores[:, 1:] = 0.0, -math.inf
        s.update(logits=wide[:, :, :V], scores=scores, done=(torch.rand(B, K, generator=gen, device="cuda") < case["done"]).to(torch.uint8),
                 eos=V // 3, out_scores=torch.empty(B, N, device="cuda"), tokens=torch.empty(B, N, dtype=torch.int32, device="cuda"),
                 parents=torch.empty(B, N, dtype=torch.int32, device="cuda"))
        if own:
            _handle(s, 1, 1, 1, 1)
            size = s["osc"].oscar_beam_select_workspace_size(B, K, V, N)
            s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    else:
        B, K, P = case["batch"], case["beams"], case["page"]
        parents, n = _family(case)
        per_req, slots = int(n.max()) // P + 2, B * K + 1
        bt = np.full((B * K, per_req), -1, np.int32)
        for b in range(B):
            k = int(n[b, 0]) // P
            bt[b * K:(b + 1) * K, :k] = rng.integers(0, 1 << 16, k)     # a prompt's pages, then some of each beam's own
            bt[b * K:(b + 1) * K, max(0, k - 2):k] = rng.integers(0, 1 << 16, (K, min(k, 2)))
        s.update(parents=dev(parents), n=dev(n.reshape(-1)), slot=dev(rng.permutation(slots)[:B * K]), bt=dev(bt),
                 tail=_slab(case, case["layers"], slots, gen), bt2=torch.empty(B * K, per_req, dtype=torch.int32, device="cuda"),
                 n2=torch.empty(B * K, dtype=torch.int32, device="cuda"), slot2=torch.empty(B * K, dtype=torch.int32, device="cuda"))
        if own:
            s["pool"] = torch.zeros(case["layers"], 1, case["kv_heads"], _sections(case)[-1], dtype=torch.uint8, device="cuda")
            _handle(s, case["layers"], slots, 1, per_req)
    return s


# ------------------------------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    if not own:
        return {"shared": _plain_shared, "beam": _plain_beam, "reorder": _plain_reorder}[case["op"]](s)
    o = s["osc"]
    if case["op"] == "shared":
        o.oscar_kv8_shared_decode_attn(s["ctx"], 0, s["q"], s["dt"], s["out"], s["odt"], s["starts"], s["shared"],
                                       len(s["sizes"]), s["most_shared"], s["bt"], s["bt"].shape[1], s["n"], s["slot"],
                                       s["n"].shape[0], s["most_own"], s["ws"], s["ws"].numel())
        return s["out"]
    if case["op"] == "beam":
        o.oscar_beam_select(s["ctx"], s["logits"], s["dt"], s["scores"], s["done"], s["eos"], case["batch"], case["beams"],
                            case["vocab"], case["n_out"], s["out_scores"], s["tokens"], s["parents"], s["ws"], s["ws"].numel())
        return {"scores": s["out_scores"], "tokens": s["tokens"], "parents": s["parents"]}
    o.oscar_kv8_reorder(s["ctx"], s["parents"], case["batch"], case["beams"], s["bt"], s["bt"].shape[1], s["n"], s["slot"],
                        s["bt2"], s["n2"], s["slot2"])
    return {"tail": s["tail"], "table": s["bt2"], "lens": s["n2"], "slots": s["slot2"]}


# ------------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "shared":
        P, d, heads = case["page"], case["d"], case["kv_heads"]
        sizes, shared, n = _grouping(case)
        page = heads * (2 * P * d + 8)
        pages = int(shared.sum()) + int(np.maximum(n // P - np.repeat(shared, sizes), 0).sum())
        q = case["q_heads"] * d * (DT[case["dtype"]].itemsize + DT[case["out"]].itemsize)
        return {"bytes": pages * page + int((n % P).sum()) * heads * 4 * d + len(n) * q, "flops": 4 * d * case["q_heads"] * int(n.sum())}
    if case["op"] == "beam":
        rows = case["batch"] * case["beams"]
        x = rows * (1 - case["done"]) * case["vocab"]
        return {"bytes": x * DT[case["dtype"]].itemsize + 5 * rows + 12 * case["batch"] * case["n_out"], "flops": 4 * x}
    parents, n = _family(case)
    row = case["layers"] * case["kv_heads"] * 2 * case["d"] * 2
    copied = sum(int(n[b, 0]) % case["page"] * (int((p >= 0).sum()) - len(set(p[p >= 0].tolist()))) for b, p in enumerate(parents))
    return {"bytes": 2 * copied * row + 8 * parents.size * (int(n.max()) // case["page"] + 5), "flops": 0}


# ------------------------------------------------------------------------------------------------- exact
def _code_table(fmt):
    b = np.arange(256)
    if fmt == "int8":
        return b - 128.0
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    return np.where(b >> 7 == 1, -v, v)


def _exact_shared(case, s):
    """Request by request over all of its pages: no grouping."""
    P, d, heads, G = case["page"], case["d"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    value = torch.from_numpy(_code_table(case["fmt"])).cuda()
    t, c = np.meshgrid(np.arange(P), np.arange(d), indexing="ij")
    flat = t * d + c
    place = []
    for i in range(2):
        turn = 2 * ((t // 2) % 4) if i else (4 * (t % 2) if d == 128 else 0 * t)
        place.append(torch.from_numpy((flat // 128 * 128 + (((flat % 128) // 16) ^ turn) * 16 + flat % 16).reshape(-1)).cuda())
    n, slot, bt = (s[x].cpu().numpy() for x in ("n", "slot", "bt"))
    out = torch.zeros(len(n), heads * G, d, dtype=torch.float64, device="cuda")
    for b in range(len(n)):
        pages, r = int(n[b]) // P, int(n[b]) % P
        mine = s["pool"][0][torch.from_numpy(bt[b, :pages].astype(np.int64)).cuda()]            # [pages, heads, size]
        scale = mine[..., 2 * P * d:2 * P * d + 8].contiguous().view(torch.float32).double()
        for h in range(heads):
            rows = s["tail"][0, int(slot[b]), h, :, :r].double()
            k, v = (torch.cat([(value[mine[:, h, i * P * d:(i + 1) * P * d][:, place[i]].int()].reshape(pages, P, d)
                                * scale[:, h, i, None, None]).reshape(-1, d), rows[i]]) for i in range(2))
            if len(k):
                w = torch.softmax(s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d), dim=1)
                out[b, h * G:(h + 1) * G] = w @ v
    return out


def exact(case, seed):
    if case["op"] == "shared" and int(_grouping(case)[2].sum()) * case["kv_heads"] * case["d"] > 3e9:
        return None
    s = prepare_plain(case, seed)
    if case["op"] == "shared":
        return _exact_shared(case, s)
    if case["op"] == "beam":
        B, N, V = case["batch"], case["n_out"], case["vocab"]
        got = np.full((B, N), -np.inf)
        for b in range(B):
            best = []
            for k in range(case["beams"]):
                start = float(s["scores"][b, k])
                if s["done"][b, k]:
                    best.append(np.array([start]))
                else:
                    x = s["logits"][b, k].double().cpu().numpy()
                    x = x[x > -np.inf]
                    if len(x):
                        part = np.sort(x)[::-1][:N]
                        best.append(start + (part - x.max()) - np.log(np.exp(x - x.max()).sum()))
            best = np.sort(np.concatenate(best))[::-1][:N] if best else np.zeros(0)
            got[b, :len(best)] = best
        return {"scores": torch.from_numpy(got).cuda(), "tokens": None, "parents": None}
    parents, n = _family(case)
    slot, tail = s["slot"].cpu().numpy().reshape(parents.shape), s["tail"].double()
    for b, p in enumerate(parents):
        kept, free = set(), [k for k in range(case["beams"]) if k not in p]
        for j, k in enumerate(p):
            if k >= 0 and k not in kept:
                kept.add(k)
                continue
            to, r = slot[b, free.pop(0)], int(n[b, 0]) % case["page"]
            if k >= 0:
                tail[:, to, :, :, :r] = tail[:, slot[b, k], :, :, :r]
    return {"tail": tail, "table": None, "lens": None, "slots": None}


def prepare_plain(case, seed):
    """The inputs of a case alone, without the context that the library's calls need."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept
