"""Operators over a cache held in 8-bit integers with one scale per page and head, and the copying and forking of
pages, measured: what is measured, in which sizes, their plain forms, and their definitions in 64 bits.

  append   new tokens' K and V quantised into the pages of an INT8 cache: a page of a head has one scale, a power
           of two, that grows when a new row needs it (the page's older codes are then rounded again)
  decode   attention of one query per sequence over an INT8 cache
  prefill  causal attention of a chunk of queries per sequence over an INT8 cache
  copy     pages copied inside a pool (any format), whole or their first rows
  fork     sequences that continue others: their block tables, and a copy of the half-filled last page
"""
import math

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ the cases

def _append(name, **kw):
    c = dict(op="append", batch=1, new=1, past=0, hkv=8, d=128, bs=16, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn(name, op, **kw):
    c = dict(op=op, batch=1, new=1, lo=4096, hi=4096, hq=32, hkv=8, d=128, bs=16, dtype="bf16", empty=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _copy(name, **kw):
    c = dict(op="copy", pages=64, partial=False, hkv=8, d=128, bs=16, cache="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _fork(name, **kw):
    c = dict(op="fork", parents=1, children=4, lo=1000, hi=1000, hkv=8, d=128, bs=16, cache="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a serving batch's decode step: one token a sequence into half-filled pages
        _append("append_step_b64", batch=64, past=2000),
        # four prompts of 2048 tokens in one call
        _append("append_prompt_4x2048", batch=4, new=2048),
        # a ragged prompt behind a few cached tokens, many heads, pages of 64
        _append("append_ragged_bs64", batch=3, new=1367, past=5, hkv=32, bs=64, dtype="f16"),
        # one request decoding: latency
        _attn("decode_b1", "decode"),
        # the 7B-like decode batch (32 heads, contexts of 1024 to 8192)
        _attn("decode_7b_b16", "decode", batch=16, lo=1024, hi=8192, hkv=32, dtype="f16"),
        # a mixed serving batch: grouped heads, contexts from 16 to 8192, one of them empty
        _attn("decode_mixed_b64", "decode", batch=64, lo=16, hi=8192, bs=32, empty=True),
        # a chunk of four long prompts, 512 queries each behind 7680 cached tokens
        _attn("prefill_chunk_4x512", "prefill", batch=4, new=512, lo=8192, hi=8192, hkv=32),
        # ragged chunks of a serving batch: grouped heads, whole prompts among them
        _attn("prefill_ragged_b3", "prefill", batch=3, new=1367, lo=1367, hi=5000, bs=32, dtype="f16"),
        # a preempted batch's pages moved: 2048 pages of a 16-bit cache
        _copy("copy_2048_pages", pages=2048),
        # copy on write: the first rows of 64 pages of an INT8 cache
        _copy("copy_int8_partial", partial=True, cache="int8"),
        # one prompt continued four ways
        _fork("fork_1_to_4"),
        # a beam step: 16 requests with 4 beams each, over an INT8 cache
        _fork("fork_beams_64", parents=64, children=64, lo=100, hi=4096, bs=32, cache="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "prefill", "prefill", "copy", "fork"))
    bs = rng.choice((8, 16, 16, 32, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    d = rng.choice((64, 128, 128))
    if op == "append":
        hkv = rng.choice((1, 3, 8, 32))
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 4096 * 32 * 128 // (batch * hkv * d)))
        return _append(None, batch=batch, new=new, past=rng.randrange(3000), hkv=hkv, d=d, bs=bs, dtype=dtype)
    if op in ("decode", "prefill"):
        hq, hkv = rng.choice(((32, 32), (32, 8), (16, 8), (8, 1), (12, 4), (40, 8), (32, 2)))
        batch = _log(rng, 1, 64 if op == "decode" else 8)
        if op == "decode":
            hi = _log(rng, 1, min(60000, 16 * 4600 * 32 * 128 // (batch * hkv * d), 16 * 4600 * 32 * 4 // (batch * hq)))
            new = 1
        else:
            new = _log(rng, 1, 2000)
            most = 4 * 512 * 7900 * 32 * 128 // (batch * new * hq * d)
            new = min(new, max(1, most))
            hi = max(new, _log(rng, new, max(new + 1, min(most, 16000))))
        return _attn(None, op, batch=batch, new=new, lo=max(new, int(hi * rng.uniform(0.05, 1.0))), hi=hi, hq=hq, hkv=hkv,
                     d=d, bs=bs, dtype=dtype, empty=op == "decode" and batch > 1 and rng.random() < 0.3)
    cache = rng.choice(("f16", "bf16", "fp8", "int8", "int8"))
    hkv = rng.choice((1, 3, 8, 32))
    page = 2 * hkv * bs * d * 2
    if op == "copy":
        return _copy(None, pages=_log(rng, 1, max(2, (1 << 27) // page)), partial=rng.random() < 0.5, hkv=hkv, d=d, bs=bs,
                     cache=cache)
    parents = _log(rng, 1, 64)
    hi = _log(rng, 1, 4096)
    return _fork(None, parents=parents, children=_log(rng, 1, 128), lo=max(1, int(hi * rng.uniform(0.05, 1.0))), hi=hi,
                 hkv=hkv, d=d, bs=bs, cache=cache)


# ------------------------------------------------------------------------------------ the inputs

def _spread(n, lo, hi, empty=False):
    """Context lengths between lo and hi, spread over their logarithm; the first is hi."""
    lens = [int(round(hi * (lo / hi) ** ((b * 0.6180339887) % 1.0))) for b in range(n)]
    if empty and n > 1:
        lens[1] = 0
    return lens


def _lens_new(case):
    """New tokens of each sequence: equal, or (several, more than a few) ragged."""
    b, n = case["batch"], case["new"]
    return [n] * b if n < 8 or n % 8 == 0 else [n - (i * 5) % 8 for i in range(b)]


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


def _int8_pool(shape, gen):
    """Codes of normal values (one in a few thousand at the end of the range) and powers of two around 2^-5."""
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - i),) + shape[1:], generator=gen, device="cuda", dtype=torch.float32)
        codes[i:i + step] = (x * 36.0).round().clamp(-127.0, 127.0).to(torch.int8)
    e = torch.randint(-6, -3, shape[:3], generator=gen, device="cuda")
    return codes, torch.ldexp(torch.ones(shape[:3], device="cuda"), e)


def _pool(kind, shape, gen):
    if kind == "int8":
        return _int8_pool(shape, gen)
    if kind == "fp8":
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * 100.0
        scales = torch.rand(shape[:4], generator=gen, device="cuda", dtype=torch.float32) * 0.02 + 0.002
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scales
    return _randn(shape, DTYPE[kind], gen), None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bs, d, hkv = case["bs"], case["d"], case["hkv"]
    s = {"op": case["op"]}
    if case["op"] == "append":
        dt, lens = DTYPE[case["dtype"]], _lens_new(case)
        start = case["past"] % (4 * bs)  # (the pages before these are not touched)
        s["table"], pages = _pages([start + n for n in lens], bs, gen)
        s["cache"], s["scales"] = _int8_pool((pages, 2, hkv, bs, d), gen)
        s["k"], s["v"] = (_randn((sum(lens), hkv, d), dt, gen) for _ in range(2))
        s["cu"], s["before"] = _cu(lens), _ints([start] * case["batch"])
    elif case["op"] in ("decode", "prefill"):
        dt = DTYPE[case["dtype"]]
        lens = _spread(case["batch"], case["lo"], case["hi"], case["empty"])
        s["table"], pages = _pages(lens, bs, gen)
        s["cache"], s["scales"] = _int8_pool((pages, 2, hkv, bs, d), gen)
        s["lens"] = _ints(lens)
        rows = [1] * case["batch"] if case["op"] == "decode" else _lens_new(case)
        s["q"] = _randn((sum(rows), case["hq"], d), dt, gen)
        s["cu"], s["most"], s["host"] = _cu(rows), max(rows), (rows, lens)
    elif case["op"] == "copy":
        n = case["pages"]
        s["cache"], s["scales"] = _pool(case["cache"], (2 * n, 2, hkv, bs, d), gen)
        order = torch.randperm(2 * n, generator=gen, device="cuda").to(torch.int32)
        s["src"], s["dst"] = order[:n].contiguous(), order[n:].contiguous()
        s["rows"] = None
        if case["partial"]:
            s["rows"] = torch.randint(0, bs + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        n, m = case["parents"], case["children"]
        lens = _spread(n, case["lo"], case["hi"])
        s["table"], pages = _pages(lens, bs, gen)
        s["cache"], s["scales"] = _pool(case["cache"], (pages + m, 2, hkv, bs, d), gen)
        s["lens"] = _ints(lens)
        s["parents"] = torch.randint(0, n, (m,), generator=gen, device="cuda", dtype=torch.int32)
        s["fresh"] = torch.arange(pages, pages + m, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------------------------------ the operators

def run(s):
    if own:
        import paged_kv_flash_cache_gb300 as pkv
        if s["op"] == "append":
            pkv.kv_cache_append(s["cache"], s["k"], s["v"], s["cu"], s["before"], s["table"], scales=s["scales"])
            return [s["cache"], s["scales"]]
        if s["op"] == "decode":
            lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
            out = pkv.paged_attn_decode(s["cache"], s["q"], s["table"], s["lens"], lse=lse, scales=s["scales"])
            return [out, lse]
        if s["op"] == "prefill":
            lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
            out = pkv.paged_attn_prefill(s["cache"], s["q"], s["cu"], s["lens"], s["table"], max_q_len=s["most"], lse=lse,
                                         scales=s["scales"])
            return [out, lse]
        if s["op"] == "copy":
            pkv.kv_cache_copy(s["cache"], s["src"], s["dst"], num_rows=s["rows"], scales=s["scales"])
            return _written(s)
        tables, lens = pkv.kv_cache_fork(s["cache"], s["table"], s["lens"], s["parents"], s["fresh"], scales=s["scales"])
        return [tables, lens] + _written(s)
    return {"append": _plain_append, "decode": _plain_attn, "prefill": _plain_attn, "copy": _plain_copy,
            "fork": _plain_fork}[s["op"]](s)


def _written(s):
    """The whole cache, and its scales."""
    return [s["cache"]] if s["scales"] is None else [s["cache"], s["scales"]]


def _power_of_two(amax):
    """The least power of two (2^-126 at least) of which 127 times are not below amax; 0 for 0."""
    m, x = torch.frexp(amax)
    e = (x - 7 + (m > 127.0 / 128.0).int()).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 0.0)


def _plain_append(s):
    cache, scales, bs = s["cache"], s["scales"], s["cache"].shape[3]
    cu, before = s["cu"].long(), s["before"].long()
    rows = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    pos = before[b] + rows - cu[b]
    page, off = s["table"][b, pos // bs].long(), pos % bs
    kv = torch.stack((s["k"], s["v"]), 1).float()                          # [T, 2, Hkv, D]
    need = torch.zeros_like(scales).index_reduce_(0, page, kv.abs().amax(-1), "amax")
    old = scales.clone()
    first = page[cu[:-1]]                                                  # the page each sequence begins in
    older = (before % bs)                                                  # its rows that are there already
    kept = torch.zeros_like(scales)
    kept[first] = torch.where(older[:, None, None] > 0, old[first], 0.0)
    scales[page] = torch.where(need > 127.0 * kept, _power_of_two(need), kept)[page]
    ratio = torch.where(scales[first] > 0, kept[first] / scales[first], 0.0)
    again = torch.round(cache[first].float() * ratio[..., None, None]).to(torch.int8)
    is_older = (torch.arange(bs, device="cuda") < older[:, None])[:, None, None, :, None]
    cache[first] = torch.where(is_older, again, cache[first])
    step = scales[page][..., None]
    cache[page, :, :, off] = torch.where(step > 0, torch.round(kv / step), 0.0).to(torch.int8)
    return [cache, scales]


def _plain_attn(s):
    cache, scales, table = s["cache"], s["scales"], s["table"]
    hkv, bs, d = cache.shape[2:]
    total, hq = s["q"].shape[:2]
    group = hq // hkv
    out, lses, at = [], [], 0
    for b, (n, length) in enumerate(zip(*s["host"])):
        q = s["q"][at:at + n].float().reshape(n, hkv, group, d)
        at += n
        pages = table[b, :-(-length // bs)].long()
        kv = cache[pages].float() * scales[pages][..., None, None]         # [pages, 2, Hkv, bs, D]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :length]
        score = torch.einsum("nhgd,hpd->hgnp", q, kv[0]) / math.sqrt(d)
        sees = torch.arange(length, device="cuda") <= torch.arange(length - n, length, device="cuda")[:, None]
        score = score.masked_fill(~sees, -math.inf) if n > 1 else score
        if length == 0:
            out.append(torch.zeros((n, hq, d), device="cuda"))
            lses.append(torch.full((n, hq), -math.inf, device="cuda"))
            continue
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - top)
        sum_p = p.sum(-1, keepdim=True)
        out.append(torch.einsum("hgnp,hpd->nhgd", p / sum_p, kv[1]).reshape(n, hq, d))
        lses.append((top + torch.log(sum_p))[..., 0].permute(2, 0, 1).reshape(n, hq))
    return [torch.cat(out).to(s["q"].dtype), torch.cat(lses)]


def _rows_to(s, src, dst, rows):
    """The first rows[i] rows of page src[i] (None: all) to page dst[i], with their scales."""
    pool = s["cache"] if s["cache"].dtype != torch.float8_e4m3fn else s["cache"].view(torch.uint8)
    if rows is None:
        pool[dst] = pool[src]
        if s["scales"] is not None:
            s["scales"][dst] = s["scales"][src]
        return
    moved = torch.arange(pool.shape[3], device="cuda") < rows[:, None]
    pool[dst] = torch.where(moved[:, None, None, :, None], pool[src], pool[dst])
    if s["scales"] is not None:
        mask = moved[:, None, None] if s["scales"].dim() == 4 else (rows > 0)[:, None, None]
        s["scales"][dst] = torch.where(mask, s["scales"][src], s["scales"][dst])


def _plain_copy(s):
    _rows_to(s, s["src"].long(), s["dst"].long(), s["rows"])
    return _written(s)


def _plain_fork(s):
    bs, parents = s["cache"].shape[3], s["parents"].long()
    lens = s["lens"][parents]
    full = lens // bs
    slot = torch.arange(s["table"].shape[1], device="cuda")
    tables = torch.where(slot < full[:, None], s["table"][parents], -1)
    tables = torch.where(slot == full[:, None], s["fresh"][:, None], tables)
    last = s["table"][parents, full.long()].clamp(min=0).long()
    _rows_to(s, last, s["fresh"].long(), lens % bs)
    return [tables, lens] + _written(s)


# ------------------------------------------------------------------------------------ what a pass needs

def work(case):
    d, hkv, bs = case["d"], case["hkv"], case["bs"]
    if case["op"] == "append":
        total = sum(_lens_new(case))
        pages = sum(-(-(case["past"] % (4 * bs) + n) // bs) - case["past"] % (4 * bs) // bs for n in _lens_new(case))
        return {"bytes": total * 2 * hkv * d * 3 + pages * 2 * hkv * 4, "flops": total * 2 * hkv * d * 2}
    if case["op"] in ("decode", "prefill"):
        lens, hq = _spread(case["batch"], case["lo"], case["hi"], case["empty"]), case["hq"]
        rows = [1] * case["batch"] if case["op"] == "decode" else _lens_new(case)
        seen = sum(n * (x - n) + n * (n + 1) // 2 if x else 0 for n, x in zip(rows, lens))
        b = sum(lens) * 2 * hkv * d + sum(-(-x // bs) for x in lens) * (2 * hkv * 4 + 4) + sum(rows) * hq * (d * 4 + 4)
        return {"bytes": b, "flops": 4 * d * hq * seen}
    size = {"f16": 2, "bf16": 2, "fp8": 1, "int8": 1}[case["cache"]]
    row = 2 * hkv * (d * size + (4 if case["cache"] == "fp8" else 0))
    page = 2 * hkv * 4 if case["cache"] == "int8" else 0
    if case["op"] == "copy":
        rows = bs / 2 if case["partial"] else bs  # (half of a page's rows on average)
        return {"bytes": int(case["pages"] * (2 * (rows * row + page) + 8)), "flops": 0}
    lens = _spread(case["parents"], case["lo"], case["hi"])
    mean = sum(x % bs for x in lens) / len(lens), sum(x // bs for x in lens) / len(lens)
    return {"bytes": int(case["children"] * (2 * (mean[0] * row + page) + 8 * mean[1] + 16)), "flops": 0}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    bs, d, hkv = case["bs"], case["d"], case["hkv"]
    if case["op"] == "append":
        # page by page: all rows that the call writes there, the scale they and the older rows ask for
        pool, scales = s["cache"].double(), s["scales"].double()
        table, start = s["table"].cpu().tolist(), s["before"].cpu().tolist()
        cu = s["cu"].cpu().tolist()
        for b in range(case["batch"]):
            at, end = start[b], start[b] + cu[b + 1] - cu[b]
            while at < end:
                n = min(bs - at % bs, end - at)
                page, off = table[b][at // bs], at % bs
                lo = cu[b] + at - start[b]
                for i, x in enumerate((s["k"], s["v"])):
                    x = x[lo:lo + n].double().transpose(0, 1)              # [Hkv, n, D]
                    most = x.abs().amax((1, 2))
                    least = torch.pow(2.0, torch.ceil(torch.log2(most.clamp(min=2.0 ** -140) / 127.0)).clamp(min=-126))
                    if off == 0:
                        new = torch.where(most > 0, least, 0.0)
                    else:
                        new = torch.where(most > 127.0 * scales[page, i], least, scales[page, i])
                        pool[page, i, :, :off] = torch.round(pool[page, i, :, :off] * (scales[page, i] / new)[:, None, None])
                    scales[page, i] = new
                    pool[page, i, :, off:off + n] = torch.round(x / new.clamp(min=2.0 ** -126)[:, None, None])
                at += n
        return [pool, scales]
    if case["op"] in ("decode", "prefill"):
        if work(case)["flops"] > 4e12:
            return None
        hq, outs, lses = case["hq"], [], []
        cu, table = s["cu"].cpu().tolist(), s["table"].cpu().tolist()
        for b, length in enumerate(s["lens"].cpu().tolist()):
            n = cu[b + 1] - cu[b]
            if length == 0:
                outs.append(torch.zeros((n, hq, d), dtype=torch.float64, device="cuda"))
                lses.append(torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            pages = torch.tensor(table[b][:(length + bs - 1) // bs], device="cuda")
            hidden = torch.ones((n, length), dtype=torch.bool, device="cuda").triu(length - n + 1)
            o, z = [], []
            for h in range(hq):
                at = h * hkv // hq
                k, v = (s["cache"][pages, i, at].double() * s["scales"][pages, i, at].double()[:, None, None] for i in (0, 1))
                x = s["q"][cu[b]:cu[b + 1], h].double() @ k.reshape(-1, d)[:length].T * d ** -0.5
                x[hidden] = -math.inf
                z.append(torch.logsumexp(x, -1))
                o.append(torch.exp(x - z[-1][:, None]) @ v.reshape(-1, d)[:length])
            outs.append(torch.stack(o, 1))
            lses.append(torch.stack(z, 1))
        return [torch.cat(outs), torch.cat(lses)]
    return None  # bits are moved, not computed: the values themselves are compared
