"""The operators around a paged KV cache that evicts: what is timed, and their plain forms.

Three operators, in the order in which a serving step runs them:

* ``norm_rope_store``: per-head RMS norm of queries and keys and the rotation by
  position, with the K/V rows written to their pool slots;
* ``decode_weights``: decode attention over the pages that also adds each key's
  softmax weight to the sums an eviction goes by;
* ``evict``: keep the first, the last and the heaviest keys of every (sequence,
  KV head) and move them to the front of the sequence's pages.

``run`` computes an operator with elementary torch operations in 32 bits, or,
where ``own`` is true, through this package's entry points.  ``exact`` is the
definition in 64 bits, one sequence at a time.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
_package = None


def _pkv():
    global _package
    if _package is None:
        import paged_kv_cache_out_gb300
        _package = paged_kv_cache_out_gb300
    return _package


# ---------------------------------------------------------------- cases
def _store(name, tokens, heads, page_size, **kw):
    q_heads, kv_heads, head_dim = heads
    case = dict(name=name, op="norm_rope_store", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, rot_dim=head_dim, norm=True, interleaved=False, fused=True,
                decode=False, page_size=page_size, context=32768)
    case.update(kw)
    return case


def _decode(name, seqs, lo, hi, spread, heads, page_size):
    q_heads, kv_heads, head_dim = heads
    return dict(name=name, op="decode_weights", seqs=seqs, min_len=lo, max_len=hi, spread=spread,
                q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size)


def _evict(name, seqs, lo, hi, spread, heads, page_size, keep, in_place=True):
    _, kv_heads, head_dim = heads
    return dict(name=name, op="evict", seqs=seqs, min_len=lo, max_len=hi, spread=spread,
                kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, keep_percent=keep,
                first=4, recent=32, in_place=in_place)


QWEN = (16, 8, 128)    # the package's Qwen3 decode, prefill and mixed-step workloads
LLAMA = (32, 8, 64)    # its long-context workload
WIDE = (32, 4, 128)    # eight query heads per KV head, the most it supports


def listed():
    return [
        # one sequence's new token: nothing but latency
        _store("store_1", 1, QWEN, 16, decode=True),
        # the decode half of a mixed step: 256 sequences, one token each
        _store("store_256", 256, QWEN, 16, decode=True),
        # one odd prefill chunk of a model without norms, q, k and v in buffers of their own
        _store("store_1021", 1021, LLAMA, 256, norm=False, fused=False),
        # eight requests' prompts of 2048 tokens
        _store("store_16384", 16384, QWEN, 16),
        # four short sequences: latency of the split and the join
        _decode("decode_tiny", 4, 37, 513, "even", QWEN, 16),
        # a full decode batch
        _decode("decode_batch", 128, 512, 4096, "even", QWEN, 16),
        # few sequences of long context: the split over the cache's length
        _decode("decode_long", 8, 16384, 32768, "even", LLAMA, 256),
        # a continuous batch from a first token to long contexts, token-granular pages
        _decode("decode_ragged", 256, 1, 8192, "log", WIDE, 1),
        # four short sequences shrink to half
        _evict("evict_tiny", 4, 37, 513, "even", QWEN, 16, 50),
        # a full decode batch shrinks to half in place: memory is short
        _evict("evict_batch", 128, 512, 4096, "even", QWEN, 16, 50),
        # long contexts shrink to a quarter in place
        _evict("evict_long", 8, 16384, 32768, "even", LLAMA, 256, 25),
        # the cached keys belong to a shared prefix too: the kept ones go to other pages
        _evict("evict_copy", 61, 100, 5000, "log", WIDE, 1, 80, in_place=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng: random.Random):
    op = rng.choice(("norm_rope_store", "decode_weights", "evict"))
    heads = rng.choice((QWEN, LLAMA, WIDE, (8, 8, 64), (8, 1, 128), (8, 2, 64)))
    page_size = rng.choice((1, 4, 16, 64, 256))
    if op == "norm_rope_store":
        tokens = _log_int(rng, 1, 12000)
        case = _store("", tokens, heads, page_size, rot_dim=rng.choice((heads[2], heads[2] // 2)),
                      norm=rng.random() < 0.7, interleaved=rng.random() < 0.4,
                      fused=heads != LLAMA and rng.random() < 0.6, decode=tokens <= 512,
                      context=rng.choice((4096, 32768)))
    else:
        seqs = _log_int(rng, 1, 200)
        # at most 170 thousand tokens over the batch
        hi = _log_int(rng, 40, min(32768, 225000 // seqs))
        lo = rng.randint(1, hi // 2)
        spread = rng.choice(("even", "log"))
        if op == "decode_weights":
            case = _decode("", seqs, lo, hi, spread, heads, page_size)
        else:
            case = _evict("", seqs, lo, hi, spread, heads, page_size, rng.randint(10, 95),
                          in_place=rng.random() < 0.7)
    del case["name"]
    return case


def _lengths(case):
    """The batch's sequence lengths in rising order: the distribution's quantiles,
    so that the work of a case does not depend on the seed."""
    n, lo, hi = case["seqs"], case["min_len"], case["max_len"]
    at = [0.5] if n == 1 else [i / (n - 1) for i in range(n)]
    if case["spread"] == "log":
        return [round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x)) for x in at]
    return [round(lo + (hi - lo) * x) for x in at]


def _kept_lengths(case, lengths):
    return [max(1, n * case["keep_percent"] // 100) for n in lengths]


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.bfloat16)


def _prepare_store(case, seed):
    gen = _generator(seed)
    T, Hq, Hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    ps, context, R = case["page_size"], case["context"], case["rot_dim"]
    if case["fused"]:  # the three are column ranges of one projection's output
        x = _bf16(gen, T, (Hq + 2 * Hkv) * d)
        q, k, v = x[:, :Hq * d], x[:, Hq * d:(Hq + Hkv) * d], x[:, (Hq + Hkv) * d:]
        q, k, v = q.view(T, Hq, d), k.view(T, Hkv, d), v.view(T, Hkv, d)
    else:
        q, k, v = _bf16(gen, T, Hq, d), _bf16(gen, T, Hkv, d), _bf16(gen, T, Hkv, d)
    if case["decode"]:  # one token of each sequence, anywhere in its context
        positions = torch.randint(0, context, (T,), generator=gen, device=DEVICE, dtype=torch.int32)
    else:  # prompts of up to 2048 tokens after cached prefixes
        start = torch.randint(0, context - 2048, (-(-T // 2048),), generator=gen, device=DEVICE)
        i = torch.arange(T, device=DEVICE)
        positions = (start[i // 2048] + i % 2048).to(torch.int32)
    pages = -(-max(T + T // 8, 256) // ps) + 1
    out_loc = torch.randperm(pages * ps, generator=gen, device=DEVICE)[:T].to(torch.int32)
    if T > 16:
        out_loc[-3:] = -1  # rows of padding
    angle = torch.arange(context, device=DEVICE, dtype=torch.float64)[:, None] * torch.pow(
        torch.tensor(1e6, device=DEVICE, dtype=torch.float64),
        -torch.arange(0, R, 2, device=DEVICE, dtype=torch.float64) / R)
    state = dict(op=case["op"], q=q, k=k, v=v, positions=positions, out_loc=out_loc,
                 cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float(),
                 k_cache=_bf16(gen, pages, ps, Hkv, d), v_cache=_bf16(gen, pages, ps, Hkv, d),
                 q_weight=None, k_weight=None, eps=1e-6, interleaved=case["interleaved"],
                 out=torch.empty(T, Hq, d, device=DEVICE, dtype=torch.bfloat16))
    if case["norm"]:
        state["q_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEVICE)).bfloat16()
        state["k_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEVICE)).bfloat16()
    return state


def _prepare_paged(case, seed):
    """Sequences of the case's lengths in shuffled order over a shuffled pool, with the sums
    of attention weights that earlier steps left."""
    gen = _generator(seed)
    Hkv, d, ps = case["kv_heads"], case["head_dim"], case["page_size"]
    lengths = _lengths(case)
    kept = _kept_lengths(case, lengths) if case["op"] == "evict" else lengths
    order = torch.randperm(len(lengths), generator=gen, device=DEVICE).tolist()
    lengths, kept = [lengths[i] for i in order], [kept[i] for i in order]
    B, longest = len(lengths), max(lengths)
    per = [-(-n // ps) for n in lengths]
    out_per = [-(-n // ps) for n in kept] if not case.get("in_place", True) else [0] * B
    used = sum(per) + sum(out_per)
    pool = used + used // 10 + 1
    ids = torch.randperm(pool, generator=gen, device=DEVICE).to(torch.int32)

    def table(counts, ids):
        counts = torch.tensor(counts, device=DEVICE)
        column = torch.arange(max(1, int(counts.max())), device=DEVICE)
        listed = column < counts[:, None]
        t = torch.full(listed.shape, -1, device=DEVICE, dtype=torch.int32)
        t[listed] = ids[:int(counts.sum())]
        return t

    rows = B + 3  # the engine keeps more request rows than this batch has
    state = dict(op=case["op"], k_cache=_bf16(gen, pool, ps, Hkv, d), v_cache=_bf16(gen, pool, ps, Hkv, d),
                 page_table=table(per, ids),
                 seq_lens=torch.tensor(lengths, device=DEVICE, dtype=torch.int32),
                 acc=torch.rand(rows, Hkv, longest, generator=gen, device=DEVICE).pow_(4).mul_(50.0 / longest),
                 acc_rows=torch.randperm(rows, generator=gen, device=DEVICE)[:B].to(torch.int32))
    # sums of about ten steps' weights, which are 1/length on average
    state["acc"][state["acc_rows"].long()] *= longest / state["seq_lens"][:, None, None]
    if case["op"] == "evict":
        state.update(keep_lens=torch.tensor(kept, device=DEVICE, dtype=torch.int32),
                     first=case["first"], recent=case["recent"],
                     page_table_out=table(out_per, ids[sum(per):]) if sum(out_per) else state["page_table"],
                     acc_out=torch.zeros(rows, Hkv, longest, device=DEVICE),
                     kept=torch.full((B, Hkv, max(kept)), -1, device=DEVICE, dtype=torch.int32),
                     new_seq_lens=torch.zeros(B, device=DEVICE, dtype=torch.int32))
    else:
        Hq = case["q_heads"]
        state.update(q=_bf16(gen, B, Hq, d), scale=d ** -0.5, max_seq_len=longest,
                     out=torch.empty(B, Hq, d, device=DEVICE, dtype=torch.bfloat16))
    return state


def prepare(case, seed):
    return (_prepare_store if case["op"] == "norm_rope_store" else _prepare_paged)(case, seed)


# ---------------------------------------------------------------- plain forms
def _normed(x, weight, eps):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        both = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        both = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((both, rest), -1)


def _plain_store(s):
    half = s["cos_sin"].shape[1] // 2
    row = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = row[..., :half], row[..., half:]
    q = _rotated(_normed(s["q"], s["q_weight"], s["eps"]), cos, sin, s["interleaved"]).bfloat16()
    k = _rotated(_normed(s["k"], s["k_weight"], s["eps"]), cos, sin, s["interleaved"]).bfloat16()
    stored = s["out_loc"] >= 0
    slots = s["out_loc"][stored].long()
    s["k_cache"].flatten(0, 1)[slots] = k[stored]
    s["v_cache"].flatten(0, 1)[slots] = s["v"][stored]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _slots(page_table, page_size, position):
    """Pool slots of positions [B, n] (0 where the table lists no page)."""
    page = torch.gather(page_table.long(), 1, position // page_size)
    return (page * page_size + position % page_size).clamp_(min=0)


def _plain_decode(s):
    q, lengths = s["q"].float(), s["seq_lens"].long()
    ps, Hkv, d = s["k_cache"].shape[1:]
    B, Hq, _ = q.shape
    position = torch.arange(s["max_seq_len"], device=q.device)
    within = position < lengths[:, None]
    slots = _slots(s["page_table"], ps, position.expand(B, -1))
    k = s["k_cache"].flatten(0, 1)[slots].float()
    scores = torch.matmul(q.view(B, Hkv, Hq // Hkv, d), k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    scores = scores.masked_fill(~within[:, None, None], -math.inf)
    weight = torch.exp(scores - scores.amax(-1, keepdim=True))
    weight = weight / weight.sum(-1, keepdim=True)
    v = s["v_cache"].flatten(0, 1)[slots].float()
    out = torch.matmul(weight, v.permute(0, 2, 1, 3)).reshape(B, Hq, d).bfloat16()
    del v
    rows = s["acc_rows"].long()
    old = s["acc"][rows][:, :, :s["max_seq_len"]]
    newest = position == lengths[:, None] - 1
    total = torch.where(newest[:, None], 0.0, old) + weight.sum(2)
    s["acc"][rows, :, :s["max_seq_len"]] = torch.where(within[:, None], total, old)
    return dict(out=out, acc=s["acc"])


def _plain_evict(s):
    lengths = s["seq_lens"].long()[:, None]
    ps, Hkv, d = s["k_cache"].shape[1:]
    kept = torch.minimum(s["keep_lens"].long()[:, None], lengths)
    first = kept.clamp(max=s["first"])
    recent = (kept - first).clamp(max=s["recent"])
    rows = s["acc_rows"].long()
    sums = s["acc"][rows]
    position = torch.arange(sums.shape[2], device=sums.device)
    safe = (position < first) | (position >= lengths - recent)
    value = sums.masked_fill(safe[:, None], math.inf)
    value = value.masked_fill((position >= lengths)[:, None], -math.inf)
    order = torch.sort(value, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, position.expand_as(order))
    stays = rank < kept[:, None]
    b, h, source = stays.nonzero(as_tuple=True)
    target = (stays.cumsum(-1) - 1)[b, h, source]
    s["kept"][b, h, target] = source.to(torch.int32)
    s["acc_out"][rows[b], h, target] = sums[b, h, source]
    from_slot = s["page_table"].long()[b, source // ps] * ps + source % ps
    to_slot = s["page_table_out"].long()[b, target // ps] * ps + target % ps
    k, v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    k[to_slot, h] = k[from_slot, h]
    v[to_slot, h] = v[from_slot, h]
    s["new_seq_lens"].copy_(kept[:, 0])
    return dict(kept=s["kept"], new_seq_lens=s["new_seq_lens"], k_cache=s["k_cache"],
                v_cache=s["v_cache"], acc=s["acc_out"])


# ---------------------------------------------------------------- the package's calls
def _own_store(s):
    q = _pkv().qk_norm_rope_store(
        s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["out_loc"], s["k_cache"], s["v_cache"],
        q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], interleaved=s["interleaved"],
        out=s["out"])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_decode(s):
    pkv = _pkv()
    if "workspace" not in s:
        B, Hq, d = s["q"].shape
        s["workspace"] = pkv.decode_weights_workspace(B, Hq, s["k_cache"].shape[2], d, s["max_seq_len"])
    out = pkv.paged_decode_attn_weights(
        s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["scale"], s["acc"],
        s["max_seq_len"], acc_rows=s["acc_rows"], workspace=s["workspace"], out=s["out"])
    return dict(out=out, acc=s["acc"])


def _own_evict(s):
    kept, new_seq_lens = _pkv().kv_evict(
        s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["keep_lens"], s["acc"],
        s["first"], s["recent"], acc_rows=s["acc_rows"], page_table_out=s["page_table_out"],
        acc_out=s["acc_out"], kept=s["kept"], new_seq_lens=s["new_seq_lens"])
    return dict(kept=kept, new_seq_lens=new_seq_lens, k_cache=s["k_cache"], v_cache=s["v_cache"],
                acc=s["acc_out"])


_PLAIN = {"norm_rope_store": _plain_store, "decode_weights": _plain_decode, "evict": _plain_evict}
_OWN = {"norm_rope_store": _own_store, "decode_weights": _own_decode, "evict": _own_evict}


def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    d, Hkv, ps = case["head_dim"], case["kv_heads"], case["page_size"]
    if case["op"] == "norm_rope_store":
        T, Hq = case["tokens"], case["q_heads"]
        elements = T * (Hq + 2 * Hkv) * d
        return dict(bytes=2 * 2 * elements + min(T, case["context"]) * case["rot_dim"] * 4 + 8 * T,
                    flops=8 * T * (Hq + Hkv) * d)
    lengths = _lengths(case)
    total = sum(lengths)
    pages = sum(-(-n // ps) for n in lengths)
    if case["op"] == "decode_weights":
        B, Hq = case["seqs"], case["q_heads"]
        # K and V rows, the sums read and written, queries and outputs, page ids, lengths and rows
        return dict(bytes=2 * 2 * total * Hkv * d + 2 * 4 * total * Hkv + 2 * 2 * B * Hq * d + 4 * pages + 8 * B,
                    flops=4 * total * Hq * d + 5 * total * Hq)
    kept = _kept_lengths(case, lengths)
    n = sum(kept)
    # in place the first keys already lie where they belong
    moved = n - (sum(min(case["first"], m) for m in kept) if case["in_place"] else 0)
    return dict(bytes=4 * total * Hkv + 2 * 2 * 2 * moved * Hkv * d + 2 * 4 * n * Hkv + 4 * pages + 16 * case["seqs"],
                flops=total * Hkv)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_store(case, s):
    T, half = case["tokens"], case["rot_dim"] // 2
    table = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / case["head_dim"] + s["eps"]).sqrt() * weight.double()
        part = x[..., :2 * half]
        pair = part.unflatten(-1, (half, 2)) if case["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat((z.reshape(part.shape), x[..., 2 * half:]), -1)

    k_new, pool = turned(s["k"], s["k_weight"]), s["k_cache"].shape
    k, v = s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
    at = torch.arange(T, device=DEVICE)[s["out_loc"] >= 0]
    k[s["out_loc"].long()[at]] = k_new[at]
    v[s["out_loc"].long()[at]] = s["v"].double()[at]
    return dict(q=turned(s["q"], s["q_weight"]), k_cache=k.view(pool), v_cache=v.view(pool))


def _sequence_slots(table_row, page_size, n):
    return (table_row[:-(-n // page_size)].long()[:, None] * page_size
            + torch.arange(page_size, device=DEVICE)).flatten()[:n]


def _exact_decode(case, s):
    ps, Hkv = case["page_size"], case["kv_heads"]
    out, acc = torch.zeros(s["q"].shape, device=DEVICE, dtype=torch.float64), s["acc"].double()
    k, v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    for b, (n, row) in enumerate(zip(s["seq_lens"].tolist(), s["acc_rows"].tolist())):
        slots = _sequence_slots(s["page_table"][b], ps, n)
        query = s["q"][b].double().unflatten(0, (Hkv, -1))
        weight = torch.einsum("hgd,nhd->hgn", query, k[slots].double()).mul_(s["scale"]).softmax(-1)
        out[b] = torch.einsum("hgn,nhd->hgd", weight, v[slots].double()).flatten(0, 1)
        acc[row, :, n - 1] = 0
        acc[row, :, :n] += weight.sum(1)
    return dict(out=out, acc=acc)


def _exact_evict(case, s):
    ps = case["page_size"]
    pool = s["k_cache"].shape
    k_old, v_old = s["k_cache"].flatten(0, 1).clone(), s["v_cache"].flatten(0, 1).clone()
    k, v = s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
    kept, acc = s["kept"].clone(), s["acc_out"].double()
    news = []
    heads = torch.arange(case["kv_heads"], device=DEVICE)[:, None]
    for b, (n, keep, row) in enumerate(zip(s["seq_lens"].tolist(), s["keep_lens"].tolist(), s["acc_rows"].tolist())):
        keep = min(n, keep)
        first = min(case["first"], keep)
        recent = min(case["recent"], keep - first)
        heavy = s["acc"][row, :, first:n - recent].double().neg().argsort(dim=-1, stable=True)[:, :keep - first - recent] + first
        ends = torch.cat((torch.arange(first, device=DEVICE), torch.arange(n - recent, n, device=DEVICE)))
        stays = torch.cat((ends.expand(len(heads), -1), heavy), 1).sort(-1).values
        kept[b, :, :keep] = stays.to(torch.int32)
        acc[row, :, :keep] = s["acc"][row].double().gather(1, stays)
        source = _sequence_slots(s["page_table"][b], ps, n)[stays]
        target = _sequence_slots(s["page_table_out"][b], ps, keep).expand_as(source)
        k[target, heads] = k_old[source, heads].double()
        v[target, heads] = v_old[source, heads].double()
        news.append(keep)
    return dict(kept=kept, new_seq_lens=torch.tensor(news, device=DEVICE, dtype=torch.int32),
                k_cache=k.view(pool), v_cache=v.view(pool), acc=acc)


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm_rope_store": _exact_store, "decode_weights": _exact_decode, "evict": _exact_evict}[case["op"]](case, state)
