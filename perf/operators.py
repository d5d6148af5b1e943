"""The operators of the 8-bit K/V cache: what is measured, and their plain forms.

A serving cache held in 8 bits keeps each sequence's keys and values, per KV head, as groups of
16 tokens with one float32 scale per group and tensor (the group is the unit that the routing
selects).  The groups live in a pool of slots, named by a table [batch, KV heads, max_groups]
in position order; the rows of the group that is still open stay in a small tail in the input's
own type.  Three operators work on it:

  append  takes new rows of K and V into the tail, writes each group that they close in 8 bits,
          and (with summary tables) the RoPE-aware summary rows that the routing reads;
  attend  one query token's exact attention over all groups and the tail, or over the sinks,
          the window and the routed groups alone; it can add each group's attention weight to
          an accumulator;
  evict   bounds a cache: keeps the sinks, the newest groups and those with the most
          accumulated weight, in order, and frees the others' slots.

Codes of a group x[16][D] with amax = max |x| and peak = 448 (e4m3) or 127 (int8):
  inverse = f32(peak / amax), scale = f32(amax / peak), code = round_to_nearest_even(f32(x * inverse));
  amax < 2^-100 counts as zero (scale and codes 0).
"""

import math
import random
from types import SimpleNamespace

import numpy as np
import torch

own = False

GROUP = 16
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
PEAK = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attend(name, **more):
    case = dict(name=name, what="attend", batch=1, heads_q=32, heads_kv=8, head_dim=128, dtype="bf16", out="f32", format="e4m3",
                shortest=1, longest=1, gone=0, weight=False, routed=0, chunk=64, sink=1, local=4)
    return {**case, **more}


def _append(name, **more):
    case = dict(name=name, what="append", batch=1, heads_kv=8, head_dim=128, dtype="bf16", format="e4m3", shortest=1, longest=1,
                token=False, summaries=False, chunk=64, n_high=32, theta=500000.0)
    return {**case, **more}


def _evict(name, **more):
    case = dict(name=name, what="evict", batch=1, heads_kv=8, shortest=1, longest=1, keep=1, sink=4, recent=16)
    return {**case, **more}


def listed():
    return [
        # one user's short prompt: latency counts
        _attend("attend_b1_1k", shortest=937, longest=937),
        # the serving batch of the decode benchmark, every token attended
        _attend("attend_b16_32k", batch=16, shortest=32761, longest=32761),
        # long contexts in integers: what the host tier holds in host memory fits the card
        _attend("attend_b8_128k_int8", batch=8, shortest=131071, longest=131071, format="int8"),
        # a ragged batch whose groups' weights are accumulated for eviction, bfloat16 outputs
        _attend("attend_ragged_weight_b16", batch=16, shortest=2240, longest=32034, weight=True, out="bf16", gone=3),
        # wide heads, routed: the sinks, the window and 32 routed groups of each (sequence, KV head)
        _attend("attend_routed_wide_b32_64k", batch=32, heads_q=64, shortest=65500, longest=65500, routed=32),
        # many short chats at once, one of them empty
        _attend("attend_b128_short", batch=128, shortest=1, longest=2051, empty=1, format="int8"),
        # a small float32 model without shared heads
        _attend("attend_f32_d64_b4", batch=4, heads_q=8, head_dim=64, dtype="f32", shortest=333, longest=4999),
        # a 64K prompt enters the cache, with the summaries that the routing needs
        _append("append_prompt_64k", shortest=65536, longest=65536, summaries=True),
        # one token of each of 16 sequences, some of which close a group
        _append("append_token_b16", batch=16, shortest=200, longest=1000, token=True, summaries=True),
        # prompts of different lengths in one padded batch, float32 into integers
        _append("append_padded_b8_f32_int8", batch=8, dtype="f32", format="int8", head_dim=64, shortest=77, longest=5003, n_high=16),
        # the steady state of a bounded cache: one group too many in each (sequence, KV head)
        _evict("evict_step_b16", batch=16, shortest=513 * GROUP, longest=513 * GROUP + 5, keep=512),
        # 128K prompts are cut down to a bounded cache
        _evict("evict_prompt_b8_128k", batch=8, shortest=131072, longest=131072, keep=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    what = rng.choice(["attend", "attend", "append", "evict"])
    heads_kv = rng.choice([1, 2, 4, 8])
    if what == "attend":
        batch = _log(rng, 1, 128)
        # at most as many tokens over all (sequence, KV head) pairs as the largest listed case has
        longest = _log(rng, 1, max(1, min(131071, 8 * 8 * 131071 // (batch * heads_kv))))
        shared = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        case = _attend("", batch=batch, heads_kv=heads_kv, heads_q=heads_kv * shared, head_dim=rng.choice([64, 128]),
                       dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["f32", "bf16"]), format=rng.choice(["e4m3", "int8"]),
                       shortest=_log(rng, 1, longest), longest=longest, weight=rng.random() < 0.4,
                       routed=rng.choice([0, 0, 0, _log(rng, 1, 128)]), chunk=rng.choice([64, 128]), sink=rng.choice([0, 1, 2]), local=rng.choice([0, 2, 4]))
        case["gone"] = 0 if case["routed"] else rng.choice([0, 0, 5])
        if batch > 2 and rng.random() < 0.3:
            case["empty"] = 1
    elif what == "append":
        batch = _log(rng, 1, 16)
        longest = _log(rng, 1, max(1, 8 * 65536 // (batch * heads_kv)))
        token = rng.random() < 0.4
        dim = rng.choice([64, 128])
        longest = min(longest, 5000) if token else longest
        case = _append("", batch=batch, heads_kv=heads_kv, head_dim=dim, dtype=rng.choice(["bf16", "bf16", "f32"]), format=rng.choice(["e4m3", "int8"]),
                       shortest=_log(rng, 1, longest), longest=longest, token=token, summaries=rng.random() < 0.5, chunk=rng.choice([64, 128]),
                       n_high=rng.choice([0, dim // 4, dim // 2]), theta=rng.choice([10000.0, 500000.0]))
    else:
        batch = _log(rng, 1, 64)
        longest = _log(rng, 16, 131072 * 8 * 8 // (batch * heads_kv) if batch * heads_kv > 64 else 131072)
        keep = _log(rng, 1, max(1, longest // GROUP))
        sink = rng.choice([0, 1, 4])
        case = _evict("", batch=batch, heads_kv=heads_kv, shortest=_log(rng, 1, longest), longest=longest, sink=min(sink, keep), keep=keep)
        case["recent"] = min(rng.choice([0, 1, 16]), keep - case["sink"])
    del case["name"]
    return case


def _lengths(case):
    """Tokens of each sequence, the same for every seed: log-spaced from shortest to longest, shuffled, `empty` of them 0."""
    n, lo, hi = case["batch"], case["shortest"], case["longest"]
    got = [round(lo * (hi / lo) ** (i / (n - 1))) if n > 1 else hi for i in range(n)]
    for i in range(case.get("empty", 0)):
        got[i] = 0
    random.Random(n * 1000003 + hi).shuffle(got)
    return got


def _max_groups(case):
    """Table entries of one (sequence, KV head): the longest sequence's groups and a few more, in whole chunks of 128 tokens."""
    return (-(-case["longest"] // GROUP) + 3 + 7) // 8 * 8


def _quantise(x, form):
    """8-bit codes (as bytes) and scales of groups x [..., 16, D], in 32 bits."""
    x = x.float()
    amax = x.abs().amax((-2, -1))
    zero = amax < 2.0 ** -100
    safe = torch.where(zero, 1.0, amax)
    peak = torch.full_like(safe, PEAK[form])  # a tensor: torch divides by a number through its reciprocal, which rounds twice
    inverse = torch.where(zero, 0.0, peak / safe)
    scale = torch.where(zero, 0.0, safe / peak)
    code = x * inverse[..., None, None]
    code = code.round().to(torch.int8) if form == "int8" else code.to(torch.float8_e4m3fn)
    return code.view(torch.uint8), scale


def _rows(gen, dim, spread, *shape):
    """Rows as a model's K and V have them: normal, with channels of different sizes."""
    return torch.randn(*shape, dim, device=DEVICE, generator=gen) * spread


def _cache(case, gen):
    """A pool with every slot filled, a table that scatters the groups over it, and a tail."""
    bh, dim, form, kind = case["batch"] * case["heads_kv"], case["head_dim"], case["format"], TYPE[case["dtype"]]
    shape = (case["batch"], case["heads_kv"])
    s = SimpleNamespace()
    s.max_groups = _max_groups(case)
    s.n_slots = bh * s.max_groups + 5
    order = torch.randperm(s.n_slots, device=DEVICE, generator=gen)
    s.table = order[: bh * s.max_groups].to(torch.int32).view(*shape, s.max_groups).contiguous()
    s.k = torch.zeros(s.n_slots, GROUP, dim, dtype=torch.uint8, device=DEVICE)
    s.v = torch.zeros_like(s.k)
    s.k_scale = torch.zeros(s.n_slots, device=DEVICE)
    s.v_scale = torch.zeros_like(s.k_scale)
    s.spread_k = torch.exp(0.5 * torch.randn(dim, device=DEVICE, generator=gen))
    s.spread_v = torch.exp(0.3 * torch.randn(dim, device=DEVICE, generator=gen))
    s.k_tail = _rows(gen, dim, s.spread_k, *shape, GROUP).to(kind)
    s.v_tail = _rows(gen, dim, s.spread_v, *shape, GROUP).to(kind)
    s.evicted = torch.full(shape, case.get("gone", 0), dtype=torch.int32, device=DEVICE)
    return s


def _fill(case, s, gen):
    step = 1 << 15
    for at in range(0, s.n_slots, step):
        n = min(step, s.n_slots - at)
        s.k[at : at + n], s.k_scale[at : at + n] = _quantise(_rows(gen, case["head_dim"], s.spread_k, n, GROUP), case["format"])
        s.v[at : at + n], s.v_scale[at : at + n] = _quantise(_rows(gen, case["head_dim"], s.spread_v, n, GROUP), case["format"])


def _groups_of(case, rng, length):
    """Ids of the routed groups of one row: ascending, from the chunks between the sinks and the window, -1 after the last."""
    per, cur = case["chunk"] // GROUP, (length - 1) // case["chunk"]
    lo, hi = case["sink"] * per, max(0, cur - case["local"]) * per
    n = min(case["routed"], max(0, hi - lo))
    got = np.sort(rng.choice(hi - lo, n, replace=False) + lo) if n else np.zeros(0, np.int64)
    return np.concatenate([got, np.full(case["routed"] - n, -1)])


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    lengths = _lengths(case)
    shape = (case["batch"], case["heads_kv"])
    s = SimpleNamespace(case=case, plan=None)
    if case["what"] == "evict":
        s.max_groups = _max_groups(case)
        s.n_slots = shape[0] * shape[1] * s.max_groups
        s.table = torch.randperm(s.n_slots, device=DEVICE, generator=gen).to(torch.int32).view(*shape, s.max_groups).contiguous()
        s.evicted = torch.randint(0, 50, shape[:1], device=DEVICE, generator=gen).to(torch.int32)[:, None].expand(shape).contiguous()
        s.pos = torch.tensor(lengths, device=DEVICE) - 1 + GROUP * s.evicted[:, 0].long()
        # accumulated weights: most groups little, a few much, equal ones among them (a new cache has zeros)
        weight = torch.exp(2.0 * torch.randn(*shape, s.max_groups, device=DEVICE, generator=gen))
        some = torch.rand(*shape, s.max_groups, device=DEVICE, generator=gen)
        weight = torch.where(some < 0.3, (weight * 4).round() / 4, weight)
        at = torch.arange(s.max_groups, device=DEVICE)
        live = -(-torch.tensor(lengths, device=DEVICE) // GROUP)
        s.weight = torch.where(at < live[:, None, None], weight, 0.0)
        s.table_out, s.weight_out, s.evicted_out = torch.empty_like(s.table), torch.empty_like(s.weight), torch.empty_like(s.evicted)
        return s
    s.__dict__.update(_cache(case, gen).__dict__)
    s.pos = torch.tensor(lengths, device=DEVICE) - 1
    kind, dim = TYPE[case["dtype"]], case["head_dim"]
    if case["what"] == "append":
        s.n_new = 1 if case["token"] else case["longest"]
        s.counts = torch.tensor([min(n, s.n_new) for n in lengths], dtype=torch.int32, device=DEVICE)
        s.k_new = _rows(gen, dim, s.spread_k, *shape, s.n_new).to(kind)
        s.v_new = _rows(gen, dim, s.spread_v, *shape, s.n_new).to(kind)
        chunks = s.max_groups * GROUP // case["chunk"]
        s.group_sum = torch.randn(*shape, chunks, case["chunk"] // GROUP, dim, device=DEVICE, generator=gen) if case["summaries"] else None
        s.chunk_sum = torch.zeros(*shape, chunks, dim, device=DEVICE) if case["summaries"] else None
        return s
    _fill(case, s, gen)
    s.pos += GROUP * case["gone"]
    s.q = (1.5 * torch.randn(case["batch"], case["heads_q"], 1, dim, device=DEVICE, generator=gen)).to(kind)
    # the first tokens of a sequence draw much of the attention
    mean = s.q.float().view(*shape, -1, dim).mean(2)
    sink = _rows(gen, dim, s.spread_k, *shape, GROUP)
    sink[:, :, 0] = 4.0 * math.sqrt(dim) * mean / mean.norm(dim=-1, keepdim=True)
    first = s.table[:, :, 0].long()
    s.k[first], s.k_scale[first] = _quantise(sink, case["format"])
    s.weight = torch.rand(*shape, s.max_groups, device=DEVICE, generator=gen) if case["weight"] else None
    s.weight_out = torch.zeros_like(s.weight) if case["weight"] else None
    s.group_idx = None
    if case["routed"]:
        rng = np.random.default_rng(seed)
        rows = [_groups_of(case, rng, n) for n in lengths for _ in range(case["heads_kv"])]
        s.group_idx = torch.tensor(np.stack(rows), dtype=torch.int32, device=DEVICE).view(*shape, case["routed"])
    s.out = torch.empty(case["batch"], case["heads_q"], 1, dim, dtype=TYPE[case["out"]], device=DEVICE)
    s.lse = torch.empty(case["batch"], case["heads_q"], 1, device=DEVICE)
    return s


def _values(s, codes, scale, slots):
    """The float32 values that the pool's slots stand for."""
    return codes[slots].view(CODE[s.case["format"]]).float() * scale[slots][..., None, None]


def _plain_attend(s):
    case = s.case
    batch, heads_kv, dim = case["batch"], case["heads_kv"], case["head_dim"]
    shared = case["heads_q"] // heads_kv
    closed = (s.pos + 1) // GROUP - case["gone"]  # [batch]: groups in the pool
    rest = (s.pos + 1) % GROUP
    if case["routed"]:  # the sinks, the window from its first chunk to the last closed group, and the routed groups
        per = case["chunk"] // GROUP
        cur = torch.clamp(s.pos, min=0) // case["chunk"]
        first = torch.clamp(cur - case["local"], min=0) * per
        end = torch.minimum(torch.full_like(first, case["sink"] * per), first)
        fixed = torch.arange((case["sink"] + case["local"] + 1) * per, device=s.pos.device)[None]
        fixed = torch.where(fixed < end[:, None], fixed, fixed - end[:, None] + first[:, None])
        fixed = torch.where(fixed < closed[:, None], fixed, -1)
        entry = torch.cat([fixed[:, None].expand(-1, heads_kv, -1), s.group_idx.long()], 2)
    else:
        entry = torch.arange(int(-(-case["longest"] // GROUP)), device=s.pos.device)
        entry = torch.where(entry < closed[:, None], entry, -1)[:, None].expand(-1, heads_kv, -1)
    seen = entry >= 0
    slots = s.table.long().gather(2, entry.clamp(min=0))
    k = torch.cat([_values(s, s.k, s.k_scale, slots), s.k_tail.float()[:, :, None]], 2).flatten(2, 3)
    there = torch.cat([seen[..., None].expand(-1, -1, -1, GROUP),
                       (torch.arange(GROUP, device=s.pos.device) < rest[:, None])[:, None, None].expand(-1, heads_kv, -1, -1)], 2)
    there = there.flatten(2, 3)[:, :, None]
    q = s.q.float().view(batch, heads_kv, shared, dim)
    score = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    del k
    score = torch.where(there, score, -math.inf)
    top = score.amax(3, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(3, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    v = torch.cat([_values(s, s.v, s.v_scale, slots), s.v_tail.float()[:, :, None]], 2).flatten(2, 3)
    v = torch.where(there.transpose(2, 3), v, 0.0)
    out = (p @ v).view(batch, case["heads_q"], 1, dim)
    lse = (torch.log(total) + torch.where(top == -math.inf, 0.0, top)).view(batch, case["heads_q"], 1)
    s.out.copy_(out)
    s.lse.copy_(lse)
    if s.weight is None:
        return {"out": s.out, "lse": s.lse}
    # weight of each group, at its table entry; the open group's entry is the one after the last closed
    each = p.sum(2).view(batch, heads_kv, -1, GROUP).sum(3)
    add = torch.zeros(batch, heads_kv, s.max_groups + 1, device=out.device)
    last = torch.where(rest > 0, closed, s.max_groups)[:, None, None].expand(-1, heads_kv, -1)
    where = torch.cat([torch.where(seen, entry, s.max_groups), last], 2)
    add.scatter_add_(2, where, torch.where(where < s.max_groups, each, 0.0))
    count = closed + (rest > 0)
    live = torch.arange(s.max_groups, device=out.device) < count[:, None, None]
    s.weight_out.copy_(torch.where(live, s.weight + add[..., : s.max_groups], s.weight_out))
    return {"out": s.out, "lse": s.lse, "weight": s.weight_out}


def _turn(case, offset, device):
    """cos and sin of the low-frequency pairs' rotation by `offset` tokens (angles in 64 bits)."""
    pairs = case["head_dim"] // 2
    i = torch.arange(case["n_high"], pairs, device=device, dtype=torch.float64)
    angle = offset.double()[:, None] * case["theta"] ** (-2.0 * i / case["head_dim"])
    return torch.cos(angle).float(), torch.sin(angle).float()


def _mean_row(case, x, offset):
    """Mean over the rows of x [..., n, D] after each one's low pairs turned by its offset."""
    half, high = case["head_dim"] // 2, case["n_high"]
    cos, sin = _turn(case, offset, x.device)
    a, b = x[..., :half], x[..., half:]
    lo_a, lo_b = a[..., high:], b[..., high:]
    a = torch.cat([a[..., :high], lo_a * cos - lo_b * sin], -1)
    b = torch.cat([b[..., :high], lo_a * sin + lo_b * cos], -1)
    return torch.cat([a, b], -1).mean(-2)


def _plain_append(s):
    case = s.case
    batch, heads_kv, dim = case["batch"], case["heads_kv"], case["head_dim"]
    count = s.counts.long()
    begin = s.pos + 1 - count
    old = begin % GROUP  # rows of the first group that the tail holds already
    groups = -(-(GROUP - 1 + s.n_new) // GROUP) if case["token"] else -(-s.n_new // GROUP)
    at = torch.arange(groups * GROUP, device=s.pos.device) - old[:, None]
    new = at.clamp(0, s.n_new - 1)[:, None, :, None].expand(-1, heads_kv, -1, dim)
    is_old = (at < 0)[:, None, :, None]
    closes = torch.arange(1, groups + 1, device=s.pos.device) * GROUP <= (old + count)[:, None]
    entry = (begin // GROUP)[:, None] + torch.arange(groups, device=s.pos.device) - s.evicted[:, :1].long()
    slots = s.table.long().gather(2, entry.clamp(0, s.max_groups - 1)[:, None].expand(-1, heads_kv, -1))
    mask = closes[:, None].expand(-1, heads_kv, -1)
    repeat = torch.arange(groups * GROUP, device=s.pos.device) % GROUP
    open_row = (old + count) // GROUP * GROUP  # first row of the group that stays open
    row = open_row[:, None] + torch.arange(GROUP, device=s.pos.device)
    stays = ((row >= old[:, None]) & (row < (old + count)[:, None]))[:, None, :, None]
    pick = (row - old[:, None]).clamp(0, s.n_new - 1)[:, None, :, None].expand(-1, heads_kv, -1, dim)
    for src, tail, codes, scale in ((s.k_new, s.k_tail, s.k, s.k_scale), (s.v_new, s.v_tail, s.v, s.v_scale)):
        x = torch.where(is_old, tail[:, :, repeat], src.gather(2, new)).view(batch, heads_kv, groups, GROUP, dim)
        code, sc = _quantise(x, case["format"])
        codes[slots[mask]] = code[mask]
        scale[slots[mask]] = sc[mask]
        if src is s.k_new and case["summaries"]:
            _plain_summaries(s, x, begin // GROUP, closes)
        tail.copy_(torch.where(stays, src.gather(2, pick), tail))
    kind = CODE[case["format"]]
    got = {"k": s.k.view(kind), "v": s.v.view(kind), "k_scale": s.k_scale, "v_scale": s.v_scale, "k_tail": s.k_tail, "v_tail": s.v_tail}
    if case["summaries"]:
        got |= {"chunk_sum": s.chunk_sum, "group_sum": s.group_sum}
    return got


def _plain_summaries(s, x, first, closes):
    """Rows of the closed groups, and of the chunks that end with one of them (from their groups' rows)."""
    case = s.case
    heads_kv, per = case["heads_kv"], case["chunk"] // GROUP
    row = _mean_row(case, x.float(), (GROUP - 1) / 2 - torch.arange(GROUP, device=x.device, dtype=torch.float64))
    total = s.max_groups
    flat = s.group_sum.view(case["batch"], heads_kv, total, -1)
    ids = first[:, None] + torch.arange(row.shape[2], device=x.device)
    b, j = torch.nonzero(closes, as_tuple=True)
    flat[b, :, ids[b, j]] = row[b, :, j]
    ends = closes & (ids % per == per - 1)
    b, j = torch.nonzero(ends, as_tuple=True)
    chunk = ids[b, j] // per
    offset = (case["chunk"] - GROUP) / 2 - GROUP * torch.arange(per, device=x.device, dtype=torch.float64)
    s.chunk_sum[b, :, chunk] = _mean_row(case, s.group_sum[b, :, chunk], offset)


def _plain_evict(s):
    case = s.case
    keep, sink, recent, total = case["keep"], case["sink"], case["recent"], s.max_groups
    closed = ((s.pos + 1) // GROUP)[:, None, None] - s.evicted.long()[..., None]
    at = torch.arange(total, device=s.pos.device)
    held = (at < sink) | (at >= closed - recent)
    worth = torch.where(held, math.inf, s.weight)
    worth = torch.where(at < closed, worth, -math.inf)
    order = torch.argsort(worth, dim=2, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order))
    kept = (at < closed) & ((rank < keep) | (closed <= keep))
    # kept groups, then the freed slots, then the slots that were free, each in their order
    place = torch.where(kept, 0, torch.where(at < closed, 1, 2))
    order = torch.argsort(place, dim=2, stable=True)
    count = kept.sum(2, keepdim=True)
    s.table_out.copy_(s.table.gather(2, order))
    weight = torch.where(at < count, s.weight.gather(2, order), 0.0)
    opened = s.weight.gather(2, closed.clamp(max=total - 1))  # the open group's weight follows the last kept one
    weight = torch.where((at == count) & (closed < total), opened, weight)
    s.weight_out.copy_(weight)
    s.evicted_out.copy_(s.evicted + (closed - count)[..., 0])
    return {"table": s.table_out, "weight": s.weight_out, "evicted": s.evicted_out}


def _plan(s):
    """The layer, the cache's description and the workspace, as a user's program makes them once."""
    from hierarchical_sparse_attention_hga_b200 import binding as B
    case = s.case
    heads_q = case.get("heads_q", case["heads_kv"])
    dim = case.get("head_dim", 128)
    layer = B.Layer(batch=case["batch"], heads_q=heads_q, heads_kv=case["heads_kv"], head_dim=dim, chunk=case.get("chunk", 64),
                    sink_chunks=case["sink"] if case["what"] == "attend" else 1, local_chunks=case.get("local", 4),
                    topk_groups=case.get("routed", 0) or 32, n_high_pairs=case.get("n_high", dim // 4), rope_theta=case.get("theta", 500000.0),
                    dtype=B.HGA_F32 if case.get("dtype") == "f32" else B.HGA_BF16, out_dtype=B.HGA_BF16 if case.get("out") == "bf16" else B.HGA_F32)
    plan = SimpleNamespace(B=B, cfg=layer.config(), ws=None, ws_bytes=0)
    form = B.HGA_QUANT_INT8 if case.get("format") == "int8" else B.HGA_QUANT_E4M3
    part = lambda name: getattr(s, name, None)  # noqa: E731
    # a cache that never evicted has no counts of evicted groups
    evicted = s.evicted if case["what"] == "evict" or case.get("gone") else None
    plan.cache = B.quant_cache(part("k"), part("v"), part("k_scale"), part("v_scale"), part("k_tail"), part("v_tail"), s.table, s.n_slots, s.max_groups, form, evicted)
    if case["what"] == "attend":
        plan.ws_bytes = B.hga_quant_attend_workspace_size(plan.cfg, s.max_groups, case["weight"])
        plan.ws = torch.empty(max(1, plan.ws_bytes), dtype=torch.uint8, device=DEVICE)
    return plan


def run(s):
    case = s.case
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}[case["what"]](s)
    if s.plan is None:
        s.plan = _plan(s)
    p = s.plan
    if case["what"] == "attend":
        p.B.hga_quant_attend(p.cfg, p.cache, s.q, s.pos, s.out, s.lse, group_idx=s.group_idx, weight_in=s.weight, weight_out=s.weight_out,
                             workspace=p.ws, workspace_bytes=p.ws_bytes)
        return {"out": s.out, "lse": s.lse} if s.weight is None else {"out": s.out, "lse": s.lse, "weight": s.weight_out}
    if case["what"] == "append":
        p.B.hga_quant_append(p.cfg, p.cache, s.k_new, s.v_new, s.n_new, s.pos, counts=s.counts, chunk_sum=s.chunk_sum, group_sum=s.group_sum)
        kind = CODE[case["format"]]
        got = {"k": s.k.view(kind), "v": s.v.view(kind), "k_scale": s.k_scale, "v_scale": s.v_scale, "k_tail": s.k_tail, "v_tail": s.v_tail}
        if case["summaries"]:
            got |= {"chunk_sum": s.chunk_sum, "group_sum": s.group_sum}
        return got
    p.B.hga_quant_evict(p.cfg, p.cache, s.pos, case["keep"], case["sink"], case["recent"], s.weight, s.weight_out, s.table_out, s.evicted_out)
    return {"table": s.table_out, "weight": s.weight_out, "evicted": s.evicted_out}


def _attended(case, length):
    """Closed groups and tail rows that a query attends."""
    closed, rest = length // GROUP, length % GROUP
    if case["routed"] and length:
        per, cur = case["chunk"] // GROUP, (length - 1) // case["chunk"]
        first = max(0, cur - case["local"]) * per
        end = min(case["sink"] * per, first)
        closed = end + closed - first + min(case["routed"], max(0, first - case["sink"] * per))
    return closed, rest


def work(case):
    lengths, heads_kv = _lengths(case), case["heads_kv"]
    if case["what"] == "evict":  # the weights and the table of the entries in use are read and written
        moved = sum(-(-n // GROUP) for n in lengths) * heads_kv
        return {"bytes": 16.0 * moved, "flops": 4.0 * moved}
    dim, size = case["head_dim"], 2 if case["dtype"] == "bf16" else 4
    if case["what"] == "append":
        new = [1 if case["token"] else n for n in lengths]
        closed = [n // GROUP - (n - m) // GROUP for n, m in zip(lengths, new)]
        old = [(n - m) % GROUP if c else 0 for n, m, c in zip(lengths, new, closed)]
        rest = [min(m, n % GROUP) for n, m in zip(lengths, new)]
        moved = sum(2 * dim * size * (m + o + r) + c * (2 * GROUP * dim + 12) for m, o, r, c in zip(new, old, rest, closed)) * heads_kv
        flops = 4.0 * sum(closed) * GROUP * dim * heads_kv
        if case["summaries"]:
            moved += (sum(closed) + sum(n // case["chunk"] - (n - m) // case["chunk"] for n, m in zip(lengths, new))) * heads_kv * dim * 4
            flops *= 2
        return {"bytes": float(moved), "flops": flops}
    some = [_attended(case, n) for n in lengths]
    tokens = sum(c * GROUP + r for c, r in some) * heads_kv
    moved = sum(c * (2 * GROUP * dim + 12) + r * 2 * dim * size for c, r in some) * heads_kv
    moved += case["batch"] * case["heads_q"] * (dim * (size + (2 if case["out"] == "bf16" else 4)) + 4)
    moved += case["batch"] * heads_kv * case["routed"] * 4
    if case["weight"]:
        moved += 8 * sum(-(-n // GROUP) for n in lengths) * heads_kv
    return {"bytes": float(moved), "flops": 4.0 * tokens * dim * case["heads_q"] / heads_kv}


# ---- the definitions in 64 bits, one (sequence, KV head) at a time


def _decoded(form):
    """The value of each of the 256 codes, from the format's definition."""
    code = np.arange(256)
    if form == "int8":
        return torch.tensor(np.where(code < 128, code, code - 256).astype(np.float64), device=DEVICE)
    e, m = (code >> 3) & 15, code & 7
    value = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    value = np.where((code & 127) == 127, np.nan, value)
    return torch.tensor(np.where(code & 128, -value, value), device=DEVICE)


def _exact_attend(case, s):
    dim, shared, lengths = case["head_dim"], case["heads_q"] // case["heads_kv"], _lengths(case)
    value = _decoded(case["format"])
    out = torch.zeros(case["batch"], case["heads_q"], 1, dim, dtype=torch.float64, device=DEVICE)
    lse = torch.full((case["batch"], case["heads_q"], 1), -math.inf, dtype=torch.float64, device=DEVICE)
    weight = s.weight_out.double() if s.weight is not None else None
    for b, length in enumerate(lengths):
        n, r = length // GROUP, length % GROUP
        for h in range(case["heads_kv"]):
            ids = list(range(n))
            if case["routed"] and length:
                per, cur = case["chunk"] // GROUP, (length - 1) // case["chunk"]
                chosen = {int(g) for g in s.group_idx[b, h].tolist() if g >= 0}
                ids = [g for g in ids if g // per < case["sink"] or g // per >= cur - case["local"] or g in chosen]
            if not length:
                continue
            at = torch.tensor(ids, dtype=torch.long, device=DEVICE)
            slot = s.table[b, h, at].long()
            k = torch.cat([(value[s.k[slot].long()] * s.k_scale[slot].double()[:, None, None]).reshape(-1, dim), s.k_tail[b, h, :r].double()])
            v = torch.cat([(value[s.v[slot].long()] * s.v_scale[slot].double()[:, None, None]).reshape(-1, dim), s.v_tail[b, h, :r].double()])
            rows = slice(h * shared, (h + 1) * shared)
            score = s.q[b, rows, 0].double() @ k.T / math.sqrt(dim)
            lse[b, rows, 0] = torch.logsumexp(score, 1)
            p = torch.exp(score - lse[b, rows])
            out[b, rows, 0] = p @ v
            if weight is not None:
                weight[b, h, : n + (r > 0)] = s.weight[b, h, : n + (r > 0)].double()
                weight[b, h, at] += p[:, : len(ids) * GROUP].reshape(shared, -1, GROUP).sum((0, 2))
                if r:
                    weight[b, h, n] += p[:, len(ids) * GROUP :].sum()
    return {"out": out, "lse": lse} if weight is None else {"out": out, "lse": lse, "weight": weight}


def _exact_codes(x, form):
    """Codes (as the values they stand for) and scales of groups x [n, 16, D] float64; products and quotients are float32's, as the definition has them."""
    amax = x.abs().flatten(1).amax(1)
    fine = amax >= 2.0 ** -100
    safe = torch.where(fine, amax, 1.0)
    peak = torch.full_like(safe, PEAK[form])
    inverse = (peak / safe).float().double() * fine
    scale = (safe / peak).float().double() * fine
    y = (x * inverse[:, None, None]).float().double()
    if form == "int8":
        return torch.round(y), scale
    # e4m3: three bits behind the leading one, steps of 2^-9 below 2^-6
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -30))), min=-6.0) - 3.0)
    return torch.round(y / step) * step, scale


def _exact_append(case, s):
    dim, form, chunk = case["head_dim"], case["format"], case["chunk"]
    code = {"k": _decoded(form)[s.k.long()], "v": _decoded(form)[s.v.long()]}
    scale = {"k": s.k_scale.double(), "v": s.v_scale.double()}
    tail = {"k": s.k_tail.double(), "v": s.v_tail.double()}
    if case["summaries"]:
        group_sum, chunk_sum = s.group_sum.double(), s.chunk_sum.double()
    i = torch.arange(dim // 2, device=DEVICE, dtype=torch.float64)
    omega = torch.where(i < case["n_high"], 0.0, case["theta"] ** (-2.0 * i / dim))

    def centred(x, offset):  # the mean of rows, as complex pairs (d, d + D/2), each turned to the centre
        z = torch.complex(x[..., : dim // 2], x[..., dim // 2 :]) * torch.exp(1j * offset[:, None] * omega)
        z = z.mean(-2)
        return torch.cat([z.real, z.imag], -1)

    for b, length in enumerate(_lengths(case)):
        count = min(length, s.n_new)
        begin = length - count
        for h in range(case["heads_kv"]):
            for name in "kv":
                held = tail[name][b, h, : begin % GROUP]
                rows = torch.cat([held, getattr(s, name + "_new")[b, h, :count].double()])
                n = len(rows) // GROUP
                first = begin // GROUP
                if n:
                    slot = s.table[b, h, first : first + n].long()
                    x = rows[: n * GROUP].view(n, GROUP, dim)
                    code[name][slot], scale[name][slot] = _exact_codes(x, form)
                    if name == "k" and case["summaries"]:
                        per = chunk // GROUP
                        flat = group_sum[b, h].view(-1, dim)
                        flat[first : first + n] = centred(x, 7.5 - torch.arange(GROUP, device=DEVICE, dtype=torch.float64))
                        for c in range(first // per, (first + n) // per):
                            turn = (chunk - GROUP) / 2 - GROUP * torch.arange(per, device=DEVICE, dtype=torch.float64)
                            chunk_sum[b, h, c] = centred(group_sum[b, h, c], turn)
                    keep = rows[n * GROUP :]
                    tail[name][b, h, : len(keep)] = keep
                else:
                    tail[name][b, h, : len(rows)] = rows
    if form == "int8":
        code = {name: x.to(torch.int8) for name, x in code.items()}
    got = {**code, "k_scale": scale["k"], "v_scale": scale["v"], "k_tail": tail["k"], "v_tail": tail["v"]}
    if case["summaries"]:
        got |= {"chunk_sum": chunk_sum, "group_sum": group_sum}
    return got


def _exact_evict(case, s):
    table, weight, evicted = (t.cpu().numpy() for t in (s.table, s.weight, s.evicted))
    table_out, weight_out, evicted_out = table.copy(), np.zeros(weight.shape, np.float64), evicted.copy()
    for b, length in enumerate(_lengths(case)):
        n = length // GROUP
        for h in range(case["heads_kv"]):
            w = weight[b, h]
            middle = list(range(case["sink"], n - case["recent"]))
            spare = max(0, n - case["keep"])
            gone = sorted(sorted(middle, key=lambda g: (w[g], -g))[:spare])  # the least weights; among equal ones the later group goes
            kept = np.setdiff1d(np.arange(n), gone)
            table_out[b, h] = np.concatenate([table[b, h, kept], table[b, h, np.array(gone, dtype=np.int64)], table[b, h, n:]])
            weight_out[b, h, : len(kept)] = w[kept]
            if n < weight.shape[2]:
                weight_out[b, h, len(kept)] = w[n]
            evicted_out[b, h] += len(gone)
    return {"table": torch.tensor(table_out), "weight": torch.tensor(weight_out), "evicted": torch.tensor(evicted_out)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}[case["what"]](case, s)
