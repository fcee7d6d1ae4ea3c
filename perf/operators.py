"""The operators of a drafted decoding step over the paged KV cache, measured: what is measured, in
which sizes, their plain forms, and their definitions in 64 bits.

  rope     the rows between a layer's projections and its attention: RMS norm of each query and key
           head, rotary positions, queries out, keys and values into their pages
  tree     attention of a tree of drafted tokens over each sequence's paged context
  compact  the cached rows that are kept (an accepted path, a window) moved to the front of a range
"""
import math

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ the cases

def _rope(name, **kw):
    c = dict(op="rope", batch=1, new=1, past=0, hq=32, hkv=8, d=128, rot=128, interleaved=False, norm=False, fused=True,
             bs=16, dtype="bf16", fp8=False, mscale=1.0, base=10000.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _tree(name, **kw):
    c = dict(op="tree", batch=1, nodes=16, lo=4096, hi=4096, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lse=True,
             fresh=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _compact(name, **kw):
    c = dict(op="compact", batch=1, keep=4, span=16, past=1024, hkv=8, d=128, bs=16, dtype="bf16", fp8=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request decoding far into a long context: latency, and the angle of a far position
        _rope("rope_one_token", past=131071),
        # a serving batch's decode step, query and key norms on
        _rope("rope_step_b64", batch=64, past=2000, norm=True, base=1000000.0),
        # four prompts of 2048 tokens in one call
        _rope("rope_prompt_4x2048", batch=4, new=2048, norm=True),
        # a ragged prompt into an FP8 cache, half of each head rotated in pairs, long-context factor
        _rope("rope_fp8_ragged", batch=3, new=1367, past=5, hkv=32, rot=64, interleaved=True, dtype="f16", fp8=True,
              mscale=1.1386),
        # one request verifying 16 drafted tokens: latency
        _tree("tree_b1_n16"),
        # the 7B-like batch (32 heads, contexts 1024 to 8192), 64 drafted tokens each
        _tree("tree_7b_b16_n64", batch=16, nodes=64, lo=1024, hi=8192, hkv=32, dtype="f16"),
        # the mixed serving batch: grouped heads, contexts from a few tokens to 8192, an odd tree,
        # a fresh sequence that has nothing but its tree, a padded node that sees nothing
        _tree("tree_mixed_b32_n63", batch=32, nodes=63, lo=63, hi=8192, bs=32, fresh=True),
        # one very long context, a small tree: the split over the keys
        _tree("tree_long_n25", nodes=25, lo=131000, hi=131000, bs=64),
        # head_dim 256, 16 / 8 heads
        _tree("tree_d256_b8_n31", batch=8, nodes=31, lo=900, hi=4100, hq=16, d=256),
        # one request's accepted path
        _compact("accept_b1"),
        # a serving batch's accepted paths
        _compact("accept_b64", batch=64, keep=6, span=63, past=2048, bs=32),
        # the windows of eight long contexts moved up behind their first pages
        _compact("window_8x8192", batch=8, keep=8192, span=16500, past=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "tree", "tree", "compact"))
    bs = rng.choice((8, 16, 16, 32, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    if op == "rope":
        fp8 = rng.random() < 0.3
        d = rng.choice((64, 128) if fp8 else (64, 128, 128, 256))
        hq, hkv = rng.choice(((32, 32), (32, 8), (16, 8), (8, 1), (12, 3)))
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 8192 * 40 * 128 // (batch * (hq + hkv) * d * 2)))
        return _rope(None, batch=batch, new=new, past=_log(rng, 1, 100000) if batch * new < 2000 else rng.randrange(100),
                     hq=hq, hkv=hkv, d=d, rot=rng.choice((d, d, d // 2, d // 4)), interleaved=rng.random() < 0.5,
                     norm=rng.random() < 0.5, fused=rng.random() < 0.7, bs=bs, dtype=dtype, fp8=fp8,
                     mscale=rng.choice((1.0, 1.0, 1.2079)), base=rng.choice((10000.0, 500000.0)))
    if op == "tree":
        d = rng.choice((64, 128, 128, 256))
        hq, hkv = rng.choice(((32, 32), (32, 8), (16, 8), (8, 1), (12, 4), (32, 2)))
        batch = _log(rng, 1, 32)
        nodes = _log(rng, 1, 200)
        most = 32 * 8192 * 8 * 128 // (batch * hkv * d * 2)   # half the largest listed case's cached bytes
        most = min(most, 12_000_000_000 // (batch * hq * nodes * d), 60000)
        hi = max(nodes, _log(rng, 64, max(65, most)))
        return _tree(None, batch=batch, nodes=nodes, lo=max(nodes, int(hi * rng.uniform(0.1, 1.0))), hi=hi, hq=hq, hkv=hkv,
                     d=d, bs=bs, dtype=dtype, lse=rng.random() < 0.5, fresh=batch > 1 and rng.random() < 0.3)
    fp8 = rng.random() < 0.3
    d = rng.choice((64, 128) if fp8 else (64, 128, 128, 256))
    hkv = rng.choice((1, 3, 8, 32))
    batch = _log(rng, 1, 64)
    keep = _log(rng, 2, max(2, min(20000, 8 * 8192 * 8 * 128 // (batch * hkv * d * 2))))
    return _compact(None, batch=batch, keep=keep, span=2 * keep + rng.randrange(1, 40), past=rng.randrange(1, 300),
                    hkv=hkv, d=d, bs=bs, dtype=dtype, fp8=fp8)


# ------------------------------------------------------------------------------------ the inputs

def _spread(case):
    """Context lengths between lo and hi, spread over their logarithm; the first is hi."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    lens = [int(round(hi * (lo / hi) ** ((b * 0.6180339887) % 1.0))) for b in range(n)]
    if case["fresh"] and n > 1:
        lens[1] = case["nodes"]
    return lens


def _lens_new(case):
    """New tokens of each sequence of a rope case: equal, or (several, more than one token) ragged."""
    b, n = case["batch"], case["new"]
    return [n] * b if n < 8 else [n - (i * 5) % 8 for i in range(b)]


def _pages(counts, bs, gen):
    """A shuffled block table for sequences of counts tokens: (table int32 [B, MB], pages in the pool)."""
    need = [max(1, -(-c // bs)) for c in counts]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    mb, at = max(need) + 1, 0
    table = torch.full((len(need), mb), -1, dtype=torch.int32, device="cuda")
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return _ints(out)


def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _fp8_pool(shape, gen):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * 100.0
    scales = torch.rand(shape[:4], generator=gen, device="cuda", dtype=torch.float32) * 0.02 + 0.002
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scales


def _a_tree(rng, n):
    """Ancestor masks (a node sees itself and its ancestors) of a random tree of n nodes, as ints."""
    seen = []
    for i in range(n):
        p = -1 if i == 0 or rng.random() < 0.1 else rng.randrange(max(0, i - 8), i)
        seen.append((1 << i) | (seen[p] if p >= 0 else 0))
    return seen


def _words(rows, nw):
    out = []
    for m in rows:
        for w in range(nw):
            x = (m >> (32 * w)) & 0xFFFFFFFF
            out.append(x - (1 << 32) if x >= 1 << 31 else x)
    return torch.tensor(out, dtype=torch.int32).reshape(len(rows), nw).cuda()


def prepare(case, seed):
    import random
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPE[case["dtype"]]
    bs, d, hkv, batch = case["bs"], case["d"], case["hkv"], case["batch"]
    s = {"op": case["op"]}
    if case["op"] == "rope":
        lens = _lens_new(case)
        total, hq = sum(lens), case["hq"]
        # a far first position needs no cached past here: the table starts at a page of its own
        start = case["past"] % (4 * bs)
        table, pages = _pages([start + n for n in lens], bs, gen)
        shape = (pages, 2, hkv, bs, d)
        if case["fp8"]:
            s["cache"], s["scales"] = _fp8_pool(shape, gen)
        else:
            s["cache"], s["scales"] = _randn(shape, dt, gen), None
        if case["fused"]:  # views into one projection's output
            x = _randn((total, (hq + 2 * hkv) * d), dt, gen)
            q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
            s["q"], s["k"], s["v"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
        else:
            s["q"], s["k"], s["v"] = (_randn((total, h, d), dt, gen) for h in (hq, hkv, hkv))
        at = torch.cat([torch.arange(n) for n in lens])
        s["positions"] = (at + case["past"]).to(torch.int32).cuda()
        s["cu"], s["before"], s["table"] = _cu(lens), _ints([start] * batch), table
        half = torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"]
        s["inv_freq"] = (case["base"] ** -half).to(torch.float32).cuda()
        s["interleaved"], s["mscale"], s["eps"] = case["interleaved"], case["mscale"], 1e-6
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (1.0 + 0.1 * _randn((2, d), torch.float32, gen)).to(dt).unbind(0)
    elif case["op"] == "tree":
        lens, n = _spread(case), case["nodes"]
        table, pages = _pages(lens, bs, gen)
        s["cache"] = _randn((pages, 2, hkv, bs, d), dt, gen)
        s["q"] = _randn((batch * n, case["hq"], d), dt, gen)
        rows = []
        for b in range(batch):
            rows += _a_tree(rng, n)
            if case["fresh"] and b == 1:
                rows[-1] = 0  # a padded node
        s["mask"] = _words(rows, -(-n // 32))
        s["cu"], s["lens"], s["table"] = _cu([n] * batch), _ints(lens), table
        s["nodes"], s["lse"] = n, case["lse"]
    else:
        keep, span, past = case["keep"], case["span"], case["past"]
        table, pages = _pages([past + span] * batch, bs, gen)
        shape = (pages, 2, hkv, bs, d)
        if case["fp8"]:
            s["cache"], s["scales"] = _fp8_pool(shape, gen)
        else:
            s["cache"], s["scales"] = _randn(shape, dt, gen), None
        # the first row kept stays where it is, the others come from behind the range they go to
        # (so that the call can be made again on the same cache)
        order = torch.rand((batch, span - keep), generator=gen, device="cuda").argsort(1)[:, :keep - 1].sort(1).values
        src = torch.cat([torch.zeros((batch, 1), dtype=torch.int64, device="cuda"), keep + order], 1) + past
        s["keep"] = src.reshape(-1).to(torch.int32)
        s["cu"], s["to"], s["table"] = _cu([keep] * batch), _ints([past] * batch), table
    return s


# ------------------------------------------------------------------------------------ the operators

def run(s):
    if own:
        import paged_kv_flash_cache_gb300 as pkv
        if s["op"] == "rope":
            q = pkv.rope_append(s["cache"], s["q"], s["k"], s["v"], s["inv_freq"], s["cu"], s["before"], s["table"],
                                positions=s["positions"], interleaved=s["interleaved"], mscale=s["mscale"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], scales=s["scales"])
            return _written(q, s)
        if s["op"] == "tree":
            lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if s["lse"] else None
            out = pkv.paged_attn_tree(s["cache"], s["q"], s["mask"], s["cu"], s["lens"], s["table"],
                                      max_q_len=s["nodes"], lse=lse)
            return [out, lse] if s["lse"] else [out]
        pkv.kv_cache_compact(s["cache"], s["keep"], s["cu"], s["to"], s["table"], scales=s["scales"])
        return _written(None, s)
    return {"rope": _plain_rope, "tree": _plain_tree, "compact": _plain_compact}[s["op"]](s)


def _written(q, s):
    """Queries and the whole cache: its values, or its codes' values and the rows' scales."""
    return [x for x in (q, s["cache"], s["scales"]) if x is not None]


def _slots(table, b, pos, bs):
    """Page and offset of position pos of sequence b."""
    pos = pos.long()
    return table[b, pos // bs].long(), pos % bs


def _sequence_of(rows, cu):
    return torch.searchsorted(cu[1:].contiguous(), rows, right=True)


def _norm(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    y, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()  # 64 bits: positions are far
    cos, sin = (angle.cos() * s["mscale"]).float()[:, None], (angle.sin() * s["mscale"]).float()[:, None]
    q = _rotate(_norm(s["q"], s["q_weight"], s["eps"]), cos, sin, s["interleaved"]).to(s["q"].dtype)
    k = _rotate(_norm(s["k"], s["k_weight"], s["eps"]), cos, sin, s["interleaved"])
    rows = torch.arange(k.shape[0], device="cuda", dtype=torch.int32)
    b = _sequence_of(rows, s["cu"])
    page, off = _slots(s["table"], b, s["before"][b] + rows - s["cu"][b], s["cache"].shape[3])
    kv = torch.stack((k, s["v"].float()), 1)
    if s["scales"] is None:
        s["cache"][page, :, :, off] = kv.to(s["cache"].dtype)
    else:
        amax = kv.abs().amax(-1, keepdim=True)
        codes = (kv * torch.where(amax > 0, 448.0 / amax, 0.0)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s["cache"].view(torch.uint8)[page, :, :, off] = codes.view(torch.uint8)
        s["scales"][page, :, :, off] = (amax / 448.0)[..., 0]
    return _written(q, s)


def _plain_tree(s):
    pool, table = s["cache"], s["table"].clamp(min=0).long()
    (batch, mb), (_, _, hkv, bs, d) = table.shape, pool.shape
    total, hq, n = s["q"].shape[0], s["q"].shape[1], s["nodes"]
    lens, cu = s["lens"].long(), s["cu"].long()
    count = cu[1:] - cu[:-1]
    kv = pool[table].float()                                  # [B, MB, 2, Hkv, bs, D]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, batch, hkv, mb * bs, d)
    pos = torch.arange(mb * bs, device="cuda")
    at = torch.arange(n, device="cuda")
    rows = (cu[:-1, None] + at).clamp(max=total - 1)          # [B, n]
    q = s["q"][rows].float().reshape(batch, n, hkv, hq // hkv, d)
    # node j of sequence b sits at position lens - count + j
    j = pos - (lens - count)[:, None]                         # [B, P]
    bits = (s["mask"][rows][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    bits = bits.flatten(2).bool()                             # [B, n, 32 * words]
    drafted = torch.gather(bits, 2, j.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, n, -1))
    sees = ((j < 0)[:, None] | (drafted & (j >= 0)[:, None])) & (pos < lens[:, None])[:, None]   # [B, n, P]
    kv = torch.where((pos < lens[:, None])[:, None, :, None], kv, 0.0)
    score = torch.einsum("bnhgd,bhpd->bhgnp", q, kv[0]) / math.sqrt(d)
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.clamp(min=-3.0e38))
    total_p = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgnp,bhpd->bnhgd", p / total_p.clamp(min=1e-30), kv[1]).reshape(batch, n, hq, d)
    lse = (top + torch.log(total_p))[..., 0].permute(0, 3, 1, 2).reshape(batch, n, hq)
    r = torch.arange(total, device="cuda")
    b = _sequence_of(r, cu)
    out, lse = out[b, r - cu[b]].to(s["q"].dtype), lse[b, r - cu[b]]
    return [out, lse] if s["lse"] else [out]


def _plain_compact(s):
    cu, bs = s["cu"].long(), s["cache"].shape[3]
    r = torch.arange(s["keep"].shape[0], device="cuda")
    b = _sequence_of(r, cu)
    page, off = _slots(s["table"], b, s["keep"], bs)
    to_page, to_off = _slots(s["table"], b, s["to"][b] + r - cu[b], bs)
    pool = s["cache"] if s["scales"] is None else s["cache"].view(torch.uint8)
    pool[to_page, :, :, to_off] = pool[page, :, :, off]
    if s["scales"] is not None:
        s["scales"][to_page, :, :, to_off] = s["scales"][page, :, :, off]
    return _written(None, s)


# ------------------------------------------------------------------------------------ what a pass needs

def work(case):
    d, hkv, batch = case["d"], case["hkv"], case["batch"]
    if case["op"] == "rope":
        total, hq = sum(_lens_new(case)), case["hq"]
        row = hkv * (d + 4) if case["fp8"] else hkv * d * 2      # a token's K (or V) as cached
        b = total * ((2 * hq + 2 * hkv) * d * 2 + 2 * row + 8)
        flops = total * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))
        return {"bytes": b, "flops": flops}
    if case["op"] == "tree":
        lens, n, hq = _spread(case), case["nodes"], case["hq"]
        seen = sum(n * (length - n) + n for length in lens)
        b = sum(lens) * hkv * d * 4 + batch * n * hq * (d * 4 + (4 if case["lse"] else 0)) + batch * n * 4 * -(-n // 32)
        return {"bytes": b, "flops": 4 * d * hq * seen}
    row = hkv * (d + 4) if case["fp8"] else hkv * d * 2
    moved = batch * (case["keep"] - 1)
    return {"bytes": moved * 4 * row + batch * case["keep"] * 4, "flops": 0}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    bs = case["bs"]
    table = s["table"].cpu().tolist()
    cu = s["cu"].cpu().tolist()
    if case["op"] == "rope":
        def turn(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
            theta = torch.outer(s["positions"].double(), s["inv_freq"].double())
            turned = x.clone()
            half = theta.shape[1]
            first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
            second = first + (1 if case["interleaved"] else half)
            z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.full_like(theta, s["mscale"]), theta)[:, None]
            turned[..., first], turned[..., second] = z.real, z.imag
            return turned
        q, k = turn(s["q"], s["q_weight"]), turn(s["k"], s["k_weight"])
        start = s["before"].cpu().tolist()
        where = [(table[b][(start[b] + i) // bs], (start[b] + i) % bs) for b in range(case["batch"])
                 for i in range(cu[b + 1] - cu[b])]
        page, off = (torch.tensor(x, device="cuda") for x in zip(*where))
        if case["fp8"]:  # a code is a rounding's answer: no value of its own
            scales = s["scales"].double()
            scales[page, 0, :, off] = k.abs().amax(-1) / 448.0
            scales[page, 1, :, off] = s["v"].double().abs().amax(-1) / 448.0
            return [q, None, scales]
        pool = s["cache"].double()
        pool[page, 0, :, off], pool[page, 1, :, off] = k, s["v"].double()
        return [q, pool]
    if case["op"] == "tree":
        n, hq, hkv, d = case["nodes"], case["hq"], case["hkv"], case["d"]
        lens, outs, lses = s["lens"].cpu().tolist(), [], []
        words = s["mask"].cpu().tolist()
        for b, length in enumerate(lens):
            pages = torch.tensor(table[b][:-(-length // bs)], device="cuda")
            kv = s["cache"][pages].double().permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :length]
            kv = kv.repeat_interleave(hq // hkv, 1)
            hidden = torch.zeros((n, length), dtype=torch.bool)
            for i in range(n):
                m = sum((w & 0xFFFFFFFF) << (32 * x) for x, w in enumerate(words[cu[b] + i]))
                hidden[i, length - n:] = torch.tensor([not (m >> y) & 1 for y in range(n)])
            x = s["q"][cu[b]:cu[b + 1]].double().transpose(0, 1) @ kv[0].transpose(1, 2) * d ** -0.5
            x[:, hidden.cuda()] = -math.inf
            lse = torch.logsumexp(x, -1)
            p = torch.where(lse[..., None] == -math.inf, torch.zeros_like(x), torch.exp(x - lse[..., None]))
            outs.append((p @ kv[1]).transpose(0, 1))
            lses.append(lse.transpose(0, 1))
        return [torch.cat(outs), torch.cat(lses)] if case["lse"] else [torch.cat(outs)]
    return None  # rows are moved, not computed: the values themselves are compared
