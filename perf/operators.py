"""The paged key/value cache: appending tokens, reading them back and attention over it.

A pool holds pages of `page` tokens, [pages, kv_heads, page, d]; a page table lists each sequence's
pages in order.  The pool's type is bf16, fp32, or e4m3 with one power-of-two scale per token and
head (stored as a biased exponent byte): value = code * 2^(exponent - 127).  A sequence's `new`
tokens are its last ones.  Three operators:

  append     writes the new tokens' keys and values into their pages (quantising them for e4m3)
  read       copies tokens out of the pages into dense tensors
  attention  softmax(scale q k^T) v of the new tokens over all cached tokens of their sequence, every
             group of heads / kv_heads query heads sharing one key/value head; with `causal` a token
             sees no later one, with `window` > 0 only keys less than `window` positions before it

Token tensors are packed [tokens, heads, d] with the sequences one after another, or padded
[batch, heads, new, d] (rows behind a sequence's last are left as they were).
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EXP_BIAS = 127
EXP_LIMIT = 50          # scales lie between 2^-50 and 2^50
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def case(name, op, dtype, batch, heads, kv_heads, d, page, max_len, new, layout="packed", causal=True, window=0):
    c = dict(op=op, dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, d=d, page=page, max_len=max_len,
             new=new, layout=layout, causal=causal, window=window)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one generated token of a small batch enters the cache: pure latency
        case("append-token-bf16", "append", "bf16", 8, 16, 8, 128, 64, 640, 1),
        # one latent frame (30 x 52) of a video enters an 8-bit cache, and is read back for the sparse path
        case("append-frame-e4m3", "append", "e4m3", 1, 12, 12, 128, 128, 32760, 1560, layout="padded"),
        # ragged prompts enter a full-precision cache of small pages
        case("append-prompts-fp32", "append", "fp32", 6, 8, 4, 64, 16, 4608, 1003),
        # a whole cached video back as dense tensors, the input of the block statistics
        case("read-video-bf16", "read", "bf16", 1, 12, 12, 128, 64, 32760, 32760, layout="padded"),
        # ragged contexts out of an 8-bit cache of small pages
        case("read-ragged-e4m3", "read", "e4m3", 16, 16, 8, 128, 16, 4608, 4608),
        # one token of one short sequence: pure latency
        case("token-short-bf16", "attention", "bf16", 1, 16, 4, 128, 32, 577, 1),
        # token generation for a ragged batch of long contexts, five query heads to a key/value head
        case("tokens-long-bf16", "attention", "bf16", 32, 40, 8, 128, 64, 32760, 1),
        # the same from an 8-bit cache, every head with its own keys
        case("tokens-e4m3", "attention", "e4m3", 64, 24, 24, 128, 128, 4608, 1, layout="padded"),
        # the next frame of a video over all cached frames, both directions inside the frame
        case("frame-bf16", "attention", "bf16", 1, 12, 12, 128, 128, 32760, 1560, layout="padded", causal=False),
        # ragged chunks of prompts over their earlier context, small pages
        case("prompts-causal-bf16", "attention", "bf16", 5, 24, 8, 128, 16, 8192, 1024),
        # the next frame (45 x 80) of the large video over an 8-bit cache: the largest call
        case("frame-large-e4m3", "attention", "e4m3", 1, 40, 40, 128, 128, 75600, 3600, layout="padded", causal=False),
        # full precision, a sliding window, short head
        case("window-fp32", "attention", "fp32", 2, 8, 2, 64, 32, 4096, 333, window=1024),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "e4m3", "bf16", "e4m3", "fp32"])
    kv = rng.choice([1, 2, 3, 4, 8, 12, 24, 40])
    heads = kv * rng.choice([g for g in (1, 1, 2, 3, 5, 8, 16) if kv * g <= 64])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    layout = rng.choice(["packed", "padded"])
    batch, max_len = spread(rng, 1, 64), spread(rng, 1, 75600)
    kind = rng.choice(["one", "one", "few", "chunk", "chunk"])
    new = 1 if kind == "one" else spread(rng, 2, 16) if kind == "few" else spread(rng, 17, 3600)
    if op == "read":
        new = max_len
    new = min(new, max_len)
    causal = rng.random() < 0.6
    window = spread(rng, 16, 8192) if op == "attention" and rng.random() < 0.25 else 0
    flops_cap = 1e11 if dtype == "fp32" else 2e12
    # a batch that costs more than the largest listed case gets smaller until it does not
    while True:
        c = case(None, op, dtype, batch, heads, kv, d, page, max_len, new, layout, causal, window)
        w = work(c)
        big = batch * kv * max_len * d * 4 > 4e9 or batch * heads * new * max_len * 4 > 3e10
        if w["bytes"] <= 2e9 and w["flops"] <= flops_cap and not (big and op != "append"):
            return c
        if batch > 1:
            batch = max(1, batch * 2 // 3)
        else:
            max_len = max(1, max_len * 2 // 3)
            new = max_len if op == "read" else max(1, min(new * 4 // 5, max_len))


def lengths(c):
    """Tokens of each sequence, and how many of them are new."""
    def part(n, k, b):
        return n if b == 0 else 1 + int((n - 1) * ((b * k) % 1.0))
    lens = [part(c["max_len"], 0.6180339887, b) for b in range(c["batch"])]
    if c["op"] == "read":
        return lens, list(lens)
    new = [min(n, part(c["new"], 0.7548776662, b)) for b, n in enumerate(lens)]
    if c["batch"] >= 4 and c["new"] > 1:
        new[2] = 0                       # a sequence that only waits
    return lens, new


def visible(c, n, m):
    """Of a sequence of n tokens, m of them new: pairs of a token and a key that it sees, keys that any sees."""
    w = c["window"] if c["window"] else n + 1
    pairs = sum((p + 1 if c["causal"] else n) - max(0, p - w + 1) for p in range(n - m, n))
    return pairs, n - max(0, n - m - w + 1) if m else 0


def work(c):
    lens, new = lengths(c)
    size = {"bf16": 2, "fp32": 4, "e4m3": 1}[c["dtype"]]
    held = 2 * c["kv_heads"] * (c["d"] * size + (1 if c["dtype"] == "e4m3" else 0))       # a cached token
    plain = c["d"] * (4 if c["dtype"] == "fp32" else 2)                                    # a token's head, dense
    if c["op"] == "attention":
        seen = [visible(c, n, m) for n, m in zip(lens, new)]
        return {"bytes": sum(k for _, k in seen) * held + 2 * sum(new) * c["heads"] * plain,
                "flops": 4 * c["d"] * c["heads"] * sum(p for p, _ in seen)}
    moved = sum(new) * (held + 2 * c["kv_heads"] * plain)
    if c["op"] == "append" and c["dtype"] == "e4m3":
        moved *= 2                       # read back as the values it stands for
    return {"bytes": moved, "flops": sum(new) * c["kv_heads"] * c["d"] * 2}


class State:
    pass


def normal(gen, shape, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)


def quantise(x):
    """Codes (e4m3) and biased exponents of the rows of x, with the smallest power of two that keeps a row in range."""
    x = x.float()
    _, e = torch.frexp(x.abs().amax(dim=-1) / E4M3_MAX)          # f * 2^e with f in [0.5, 1)
    exact_power = torch.ldexp(torch.full_like(x[..., 0], 0.5), e) * E4M3_MAX == x.abs().amax(dim=-1)
    e = (e - exact_power.int()).clamp(-EXP_LIMIT, EXP_LIMIT)
    codes = torch.ldexp(x, -e.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, (e + EXP_BIAS).to(torch.uint8)


def token_tensors(c, gen, dev, heads, n, total, shift):
    """A tensor of the new tokens (n of a sequence at most, total in all): unit normal, a few channels shifted, as keys have."""
    shape = (total, heads, c["d"]) if c["layout"] == "packed" else (c["batch"], heads, max(1, n), c["d"])
    x = normal(gen, shape, dev)
    x[..., :: c["d"] // 4] += shift
    return x.to(TORCH["fp32" if c["dtype"] == "fp32" else "bf16"])


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, new = lengths(c)
    s = State()
    s.c, s.max_new = c, max(new)
    per_seq = [-(-n // c["page"]) for n in lens]
    s.max_pages = max(per_seq)
    pages = sum(per_seq) + 3             # a few that no sequence holds
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    at = torch.tensor([0] + per_seq).cumsum(0)[:-1]
    cols = torch.arange(s.max_pages)[None, :]
    index = (at[:, None] + cols).clamp(max=pages - 1).to(dev)
    s.page_table = order[index].contiguous()
    s.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    s.new = torch.tensor(new, dtype=torch.int32, device=dev)
    s.starts = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(dev)
    total = sum(new)
    # pools as a program finds them after use: every slot holds some token, stale ones among them
    shape = (pages, c["kv_heads"], c["page"], c["d"])
    kp, vp = normal(gen, shape, dev), normal(gen, shape, dev)
    kp[..., :: c["d"] // 4] += 1.5
    if c["dtype"] == "e4m3":
        s.k_pool, s.k_exp = quantise(kp)
        s.v_pool, s.v_exp = quantise(vp)
        s.k_pool, s.v_pool = s.k_pool.view(torch.uint8), s.v_pool.view(torch.uint8)
    else:
        s.k_pool, s.v_pool = kp.to(TORCH[c["dtype"]]), vp.to(TORCH[c["dtype"]])
        s.k_exp = s.v_exp = None
    del kp, vp
    s.scale = 1.0 / math.sqrt(c["d"])
    if c["op"] == "attention":
        s.q = token_tensors(c, gen, dev, c["heads"], s.max_new, total, 0.25)
        s.o = torch.zeros_like(s.q)
    elif c["op"] == "append":
        s.k = token_tensors(c, gen, dev, c["kv_heads"], s.max_new, total, 1.5)
        s.v = token_tensors(c, gen, dev, c["kv_heads"], s.max_new, total, 0.0)
        s.k_out, s.v_out = torch.zeros_like(s.k), torch.zeros_like(s.v)
    else:
        out = (total, c["kv_heads"], c["d"]) if c["layout"] == "packed" else (c["batch"], c["kv_heads"], s.max_new, c["d"])
        s.k_out = torch.zeros(out, dtype=TORCH["fp32" if c["dtype"] == "fp32" else "bf16"], device=dev)
        s.v_out = torch.zeros_like(s.k_out)
    if own:
        from piecewise_approximate_attention_b200.runtime import PagedCache
        s.cache = PagedCache(pages, c["heads"], c["kv_heads"], c["page"], c["d"], c["dtype"], device=dev,
                             k=s.k_pool, v=s.v_pool, k_exp=s.k_exp, v_exp=s.v_exp)
        ragged = dict(starts=s.starts) if c["layout"] == "packed" else dict(counts=s.new)
        s.seqs = s.cache.sequences(s.page_table, s.lens, max_len=c["max_len"], max_new=s.max_new, **ragged)
    return s


def run(s):
    if own:
        return run_own(s)
    return {"append": plain_append, "read": plain_read, "attention": plain_attention}[s.c["op"]](s)


def run_own(s):
    c = s.c
    if c["op"] == "attention":
        s.cache.attention(s.seqs, s.q, s.o, causal=c["causal"], window=c["window"], softmax_scale=s.scale)
        return s.o
    if c["op"] == "append":
        s.cache.append(s.seqs, s.k, s.v)
        if c["dtype"] != "e4m3":
            return s.k_pool, s.v_pool
    s.cache.read(s.seqs, s.k_out, s.v_out)
    return s.k_out, s.v_out


# ---- plain forms -------------------------------------------------------------------------------
def new_tokens(s):
    """For every new token: its sequence, its number among the new ones, its page and its slot there."""
    count = s.new.long()
    step = torch.arange(s.max_new, device=count.device)
    b, i = (step[None, :] < count[:, None]).nonzero(as_tuple=True)
    pos = s.lens.long()[b] - count[b] + i
    return b, i, s.page_table.long()[b, pos // s.c["page"]], pos % s.c["page"]


def packed_rows(s, x, b, i):
    return x if s.c["layout"] == "packed" else x[b, :, i]


def store_rows(s, out, x, b, i):
    if s.c["layout"] == "packed":
        out.copy_(x)
    else:
        out[b, :, i] = x.to(out.dtype)


def values(codes, exps):
    """What a pool's rows stand for, in 32 bits."""
    if exps is None:
        return codes.float()
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exps.int().unsqueeze(-1) - EXP_BIAS)


def plain_append(s):
    b, i, page, slot = new_tokens(s)
    k, v = packed_rows(s, s.k, b, i), packed_rows(s, s.v, b, i)
    if s.c["dtype"] != "e4m3":
        s.k_pool[page, :, slot] = k
        s.v_pool[page, :, slot] = v
        return s.k_pool, s.v_pool
    kc, ke = quantise(k)
    vc, ve = quantise(v)
    s.k_pool[page, :, slot], s.k_exp[page, :, slot] = kc.view(torch.uint8), ke
    s.v_pool[page, :, slot], s.v_exp[page, :, slot] = vc.view(torch.uint8), ve
    return plain_read(s)


def plain_read(s):
    b, i, page, slot = new_tokens(s)
    ke, ve = (None, None) if s.k_exp is None else (s.k_exp[page, :, slot], s.v_exp[page, :, slot])
    store_rows(s, s.k_out, values(s.k_pool[page, :, slot], ke), b, i)
    store_rows(s, s.v_out, values(s.v_pool[page, :, slot], ve), b, i)
    return s.k_out, s.v_out


def dense_cache(s, pool, exps):
    """[batch, kv_heads, tokens, d] in 32 bits, the sequences padded to the longest page list."""
    table = s.page_table.long()
    x = values(pool[table], None if exps is None else exps[table])      # [batch, pages, kv_heads, page, d]
    return x.transpose(1, 2).flatten(2, 3)


def plain_attention(s):
    c = s.c
    b, i, _, _ = new_tokens(s)
    group, n = c["heads"] // c["kv_heads"], s.max_new
    k, v = dense_cache(s, s.k_pool, s.k_exp), dense_cache(s, s.v_pool, s.v_exp)
    if c["layout"] == "packed":
        q = torch.zeros(c["batch"], c["heads"], n, c["d"], device=k.device)
        q[b, :, i] = s.q.float()
    else:
        q = s.q.float()
    q = q.reshape(c["batch"], c["kv_heads"], group * n, c["d"])
    logits = (q @ k.transpose(2, 3)).mul_(s.scale).view(c["batch"], c["kv_heads"], group, n, -1)
    key = torch.arange(k.shape[2], device=k.device)
    pos = (s.lens - s.new)[:, None] + torch.arange(n, device=k.device)[None, :]
    seen = (key[None, None, :] < s.lens[:, None, None]).expand(-1, n, -1)
    if c["causal"]:
        seen = seen & (key[None, None, :] <= pos[:, :, None])
    if c["window"]:
        seen = seen & (key[None, None, :] > pos[:, :, None] - c["window"])
    hidden = ~seen[:, None, None]
    logits.masked_fill_(hidden, -math.inf)
    top = logits.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = logits.sub_(top).exp_()
    norm = p.sum(dim=-1).clamp(min=1e-30).view(c["batch"], c["kv_heads"], group * n, 1)
    # stale slots hold finite numbers here, and their weight is zero
    o = (p.view(c["batch"], c["kv_heads"], group * n, -1) @ v).div_(norm).view(c["batch"], c["heads"], n, c["d"])
    if c["layout"] == "packed":
        s.o.copy_(o[b, :, i])
    else:
        s.o[b, :, i] = o[b, :, i].to(s.o.dtype)
    return s.o


# ---- the definition in 64 bits -----------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    lens, new = lengths(c)
    table = s.page_table.cpu().tolist()

    def slots(b, first, last):
        page, size = table[b], c["page"]
        return (torch.tensor([page[t // size] for t in range(first, last)], device="cuda"),
                torch.tensor([t % size for t in range(first, last)], device="cuda"))

    def held(pool, exps, b, first, last):                    # [kv_heads, tokens, d] as 64-bit numbers
        p, t = slots(b, first, last)
        x = pool[p, :, t]
        if exps is None:
            return x.double().transpose(0, 1)
        two = torch.tensor(2.0, dtype=torch.float64, device="cuda")
        return (x.view(torch.float8_e4m3fn).double() * two.pow(exps[p, :, t].double() - 127)[..., None]).transpose(0, 1)

    def rows(x, b):                                          # [heads, tokens, d] of sequence b, a view
        if c["layout"] == "packed":
            at = sum(new[:b])
            return x[at:at + new[b]].transpose(0, 1)
        return x[b, :, :new[b]]

    if c["op"] == "append":
        if c["dtype"] == "e4m3":
            return exact_rounding(s, c)
        k, v = s.k_pool.double(), s.v_pool.double()
        for b in range(c["batch"]):
            p, t = slots(b, lens[b] - new[b], lens[b])
            if new[b]:
                k[p, :, t] = rows(s.k, b).double().transpose(0, 1)
                v[p, :, t] = rows(s.v, b).double().transpose(0, 1)
        return k, v
    if c["op"] == "read":
        k, v = s.k_out.double(), s.v_out.double()
        for b in range(c["batch"]):
            rows(k, b).copy_(held(s.k_pool, s.k_exp, b, 0, lens[b]))
            rows(v, b).copy_(held(s.v_pool, s.v_exp, b, 0, lens[b]))
        return k, v
    out = torch.zeros(s.o.shape, dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    for b in range(c["batch"]):
        if not new[b]:
            continue
        n, m = lens[b], new[b]
        k, v = held(s.k_pool, s.k_exp, b, 0, n), held(s.v_pool, s.v_exp, b, 0, n)
        q, o = rows(s.q, b), rows(out, b)
        at = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None, :]
        drop = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if c["causal"]:
            drop |= j > at
        if c["window"]:
            drop |= at - j >= c["window"]
        for h in range(c["heads"]):
            a = torch.softmax((q[h].double() @ k[h // group].T * s.scale).masked_fill_(drop, -math.inf), dim=-1)
            o[h] = a @ v[h // group]
    return out


def exact_rounding(s, c):
    """Each row over its scale, rounded to three fraction bits (steps of 2^-9 below 2^-6), in 64 bits."""
    def rounded(x):
        x = x.double()
        e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / E4M3_MAX)).clamp(-EXP_LIMIT, EXP_LIMIT)
        y = x / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step * torch.exp2(e)
        if c["layout"] == "padded":      # only the sequences' own rows are returned
            y *= (torch.arange(x.shape[2], device=x.device)[None, :] < s.new[:, None])[:, None, :, None]
        return y

    return rounded(s.k), rounded(s.v)


if __name__ == "__main__":
    for n in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(n, work(n))
