"""Measured operators of a speculative-decoding step over a paged KV cache.

Three operators a serving loop calls one after the other when the new tokens
of a sequence are a tree of drafted tokens instead of a run:

  rotary   Q and K rows rotated at explicit positions with frequencies scaled
           for long contexts; K and V go to the paged pool ("paged") or Q and
           K to plain outputs;
  tree     attention of the drafted tokens over the cached context and over
           their own ancestors (a bit mask), with optional softcap, window,
           distance bias and sinks;
  commit   the accepted path's K/V rows moved to the front of the draft slots
           in every layer's pools.

`own` selects the plain torch form (False) or the library's calls (True).
Lengths, trees and tables depend on the case alone, values on the seed.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TWO_PI = 2.0 * math.pi


def listed():
    return [
        # one user, a short draft over a short context: what a single step costs at least
        dict(name="tree_one_user", kind="tree", batch=1, heads=32, kv_heads=8, head_size=128, block_size=16,
             ctx_lo=600, ctx_hi=600, draft=5, ragged=False, dtype="fp16", softcap=0.0, window=-1, bias=False,
             sink=False, lens=1),
        # a full serving batch with a small ragged tree per sequence
        dict(name="tree_batch", kind="tree", batch=64, heads=32, kv_heads=8, head_size=128, block_size=16,
             ctx_lo=512, ctx_hi=4096, draft=8, ragged=True, dtype="bf16", softcap=0.0, window=-1, bias=False,
             sink=False, lens=2),
        # wide trees of a 64-head layer: 512 query rows per kv head, where the products count
        dict(name="tree_wide", kind="tree", batch=16, heads=64, kv_heads=8, head_size=128, block_size=32,
             ctx_lo=1024, ctx_hi=8192, draft=64, ragged=False, dtype="fp16", softcap=0.0, window=-1, bias=False,
             sink=False, lens=3),
        # two very long documents, a medium tree each: few sequences, long axis
        dict(name="tree_long", kind="tree", batch=2, heads=32, kv_heads=8, head_size=128, block_size=64,
             ctx_lo=100000, ctx_hi=131072, draft=32, ragged=False, dtype="bf16", softcap=0.0, window=-1, bias=False,
             sink=False, lens=4),
        # a windowed layer with capped scores and sinks over long contexts
        dict(name="tree_window_cap", kind="tree", batch=8, heads=16, kv_heads=8, head_size=64, block_size=64,
             ctx_lo=20001, ctx_hi=32768, draft=24, ragged=True, dtype="fp16", softcap=50.0, window=4096, bias=False,
             sink=True, lens=5),
        # one kv head per query head with a distance bias, odd lengths
        dict(name="tree_bias", kind="tree", batch=32, heads=16, kv_heads=16, head_size=64, block_size=16,
             ctx_lo=1, ctx_hi=2047, draft=13, ragged=True, dtype="bf16", softcap=0.0, window=-1, bias=True,
             sink=False, lens=6),
        # the draft of one user, rotated and written to its pages
        dict(name="rotary_one_user", kind="rotary", paged=True, batch=1, heads=32, kv_heads=8, head_size=128,
             block_size=16, draft=5, ragged=False, rotary_dim=128, rotary_offset=0, interleaved=False,
             scaling="none", far=600, dtype="fp16", lens=7),
        # the drafts of a batch at far positions of a model scaled by parts
        dict(name="rotary_batch_far", kind="rotary", paged=True, batch=64, heads=64, kv_heads=8, head_size=128,
             block_size=32, draft=64, ragged=True, rotary_dim=128, rotary_offset=0, interleaved=False,
             scaling="by_parts", far=900000, dtype="bf16", lens=8),
        # a long prompt, part of each head in interleaved pairs, to plain outputs
        dict(name="rotary_prompt", kind="rotary", paged=False, batch=1, heads=32, kv_heads=8, head_size=128,
             block_size=16, draft=16385, ragged=False, rotary_dim=64, rotary_offset=0, interleaved=True,
             scaling="linear", far=120000, dtype="fp16", lens=9),
        # one sequence's accepted path, every layer of a 32-layer model
        dict(name="commit_one_user", kind="commit", layers=32, batch=1, kv_heads=8, head_size=128, block_size=16,
             draft=8, most=5, dtype="fp16", lens=19),
        # a batch's accepted paths in an 80-layer model
        dict(name="commit_batch", kind="commit", layers=80, batch=128, kv_heads=8, head_size=128, block_size=16,
             draft=32, most=12, dtype="bf16", lens=11),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "rotary", "commit"])
    limit = max(_cost(c) for c in listed() if c["kind"] == kind)
    while True:
        case = _draw_one(rng, kind)
        if _cost(dict(case, window=-1)) <= limit:  # a window shortens the reads, not the cache
            return case


def _draw_one(rng, kind):
    lens = rng.randrange(1 << 20)
    if kind == "tree":
        group = rng.choice([1, 2, 4, 5, 8, 16])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        hi = _log_int(rng, 1, 131072)
        return dict(kind="tree", batch=_log_int(rng, 1, 64), heads=group * kv_heads, kv_heads=kv_heads,
                    head_size=rng.choice([64, 128]), block_size=rng.choice([16, 32, 64, 128, 256]),
                    ctx_lo=max(0, int(hi * rng.random())), ctx_hi=hi, draft=_log_int(rng, 1, 128),
                    ragged=rng.random() < 0.7, dtype=rng.choice(["fp16", "bf16"]),
                    softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([-1, -1, _log_int(rng, 16, 8192)]),
                    bias=rng.random() < 0.25, sink=rng.random() < 0.25, lens=lens)
    if kind == "rotary":
        paged = rng.random() < 0.6
        head_size = rng.choice([64, 128, 256] if not paged else [64, 128])
        rotary_dim = rng.choice([head_size, head_size // 2, 16 * rng.randint(1, head_size // 16)])
        return dict(kind="rotary", paged=paged, batch=_log_int(rng, 1, 64) if paged else 1,
                    heads=rng.choice([8, 16, 32, 64]), kv_heads=rng.choice([1, 2, 8]), head_size=head_size,
                    block_size=rng.choice([16, 32, 64]),
                    draft=_log_int(rng, 1, 64) if paged else _log_int(rng, 1, 16385), ragged=rng.random() < 0.5,
                    rotary_dim=rotary_dim, rotary_offset=8 * rng.randint(0, (head_size - rotary_dim) // 8),
                    interleaved=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "base", "by_parts", "by_wavelength"]),
                    far=_log_int(rng, 1, 1000000), dtype=rng.choice(["fp16", "bf16"] + ([] if paged else ["fp32"])),
                    lens=lens)
    draft = _log_int(rng, 2, 64)
    return dict(kind="commit", layers=rng.choice([1, 2, 16, 32, 61, 80]), batch=_log_int(rng, 1, 128),
                kv_heads=rng.choice([1, 2, 4, 8]), head_size=rng.choice([64, 128, 256]),
                block_size=rng.choice([16, 32, 64]), draft=draft, most=rng.randint(2, max(2, min(draft, 16))),
                dtype=rng.choice(["fp16", "bf16"]), lens=lens)


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def _plan(case):
    """Lengths, trees and accepted paths: everything whole-numbered, from the case alone."""
    r = random.Random(case["lens"])
    B, n_max = case["batch"], case["draft"]
    n = [r.randint(1, n_max) if case.get("ragged") and n_max > 1 else n_max for _ in range(B)]
    if case["kind"] == "tree":
        past = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    else:
        past = [r.randint(0, 40) for _ in range(B)]
    parents, depths, paths = [], [], []
    for b in range(B):
        if case["kind"] == "rotary" and not case["paged"]:
            parents.append([])
            depths.append(list(range(n[b])))
            continue
        # node 0 is the token sampled last; a later node hangs below one of the nodes just before it
        par, dep = [-1], [0]
        for j in range(1, n[b]):
            p = r.randint(max(0, j - 6), j - 1)
            par.append(p)
            dep.append(dep[p] + 1)
        parents.append(par)
        depths.append(dep)
        if case["kind"] == "commit":
            path, j = [], max(range(n[b]), key=lambda i: (dep[i], r.random()))
            while j >= 0:
                path.append(j)
                j = par[j]
            paths.append(path[::-1][:r.randint(1, case["most"])])
    return dict(n=n, past=past, parents=parents, depths=depths, paths=paths)


def _moved(path):
    return sum(1 for i, a in enumerate(path) if a != i)


def work(case):
    plan, kind = _plan(case), case["kind"]
    e = 4 if case["dtype"] == "fp32" else 2
    if kind == "commit":
        rows = sum(_moved(p) for p in plan["paths"])
        idx = 4 * sum(len(p) for p in plan["paths"]) + 12 * case["batch"]
        return {"bytes": float(4 * rows * case["kv_heads"] * case["head_size"] * e * case["layers"] + idx),
                "flops": 0.0}
    H, Hk, D = case["heads"], case["kv_heads"], case["head_size"]
    T = sum(plan["n"])
    if kind == "rotary":
        rows = H + (2 * Hk if case["paged"] else Hk)
        return {"bytes": float(2 * T * rows * D * e + 4 * T + 4 * case["rotary_dim"]),
                "flops": float(6 * T * (H + Hk) * case["rotary_dim"] // 2)}
    kv, pairs = 0, 0
    for past, par, dep in zip(plan["past"], plan["parents"], plan["depths"]):
        W = case["window"]
        lo = max(0, past + min(dep) + 1 - W) if W > 0 else 0
        kv += max(0, past - lo) + len(par)
        for d in dep:
            pairs += max(0, past - (max(0, past + d + 1 - W) if W > 0 else 0)) + (min(d + 1, W) if W > 0 else d + 1)
    return {"bytes": float(kv * Hk * D * 2 * e + 2 * T * H * D * e), "flops": float(4 * D * H * pairs)}


def _frequencies(case):
    """Radians per position of each pair (64 bits), and the factor on cos and sin."""
    R, base, s, original = case["rotary_dim"], 10000.0, 8.0, 8192.0
    i = torch.arange(R // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "base":
        return (base * s ** (R / max(R - 2, 1))) ** (-2.0 * i / R), 1.0
    if case["scaling"] == "by_parts":
        at = [R * math.log(original / (turns * TWO_PI)) / (2.0 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f / s * ramp + f * (1.0 - ramp), 0.1 * math.log(s) + 1.0
    if case["scaling"] == "by_wavelength":
        keep = ((original * f / TWO_PI - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f / s * (1.0 - keep) + f * keep, 1.0
    return f, 1.0


def _pages(case, plan, gen):
    """A shuffled block table whose rows cover each sequence's cached and drafted slots."""
    bs = case["block_size"]
    need = [-(-(p + n) // bs) for p, n in zip(plan["past"], plan["n"])]
    total = sum(need)
    order = torch.randperm(total + max(2, total // 10), generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((case["batch"], max(need)), -1, dtype=torch.int32, device="cuda")
    rows = torch.repeat_interleave(torch.arange(case["batch"]), torch.tensor(need)).cuda()
    first = torch.cumsum(torch.tensor(need), 0) - torch.tensor(need)
    cols = torch.arange(total).cuda() - first.cuda()[rows]
    table[rows, cols] = order[:total]
    return table, order.numel()


def prepare(case, seed):
    plan, kind = _plan(case), case["kind"]
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + case["lens"])
    dtype, D = DTYPES[case["dtype"]], case["head_size"]

    def randn(*size, std=1.0):
        return torch.randn(*size, generator=gen, device="cuda", dtype=dtype).mul_(std)

    past = torch.tensor(plan["past"], dtype=torch.int32)
    n = torch.tensor(plan["n"], dtype=torch.int32)
    cum = torch.zeros(case["batch"] + 1, dtype=torch.int32)
    cum[1:] = torch.cumsum(n, 0)
    T, Hk = int(cum[-1]), case["kv_heads"]
    s = dict(case=case, T=T, past=past.cuda(), cum=cum.cuda(), n=n.cuda(), draft=case["draft"])
    depth = torch.tensor([d for row in plan["depths"] for d in row], dtype=torch.int32)
    owner = torch.repeat_interleave(torch.arange(case["batch"]), n.long())
    s["owner"] = owner.cuda()
    table = None
    if kind != "rotary" or case["paged"]:
        table, blocks = _pages(case, plan, gen)
        s["table"] = table
    if kind == "commit":
        s["pools"] = randn(case["layers"], 2, blocks, case["block_size"], Hk, D)
        width = case["most"]
        accepted = torch.tensor([p + [0] * (width - len(p)) for p in plan["paths"]], dtype=torch.int32)
        s["accepted"] = accepted.cuda()
        s["count"] = torch.tensor([len(p) for p in plan["paths"]], dtype=torch.int32).cuda()
        s["new_past"] = torch.empty_like(s["past"])
    elif kind == "rotary":
        H = case["heads"]
        start = torch.randint(0, case["far"] + 1, (case["batch"],), generator=gen, device="cuda", dtype=torch.int32)
        s["positions"] = start[s["owner"]] + depth.cuda()
        freq, s["factor"] = _frequencies(case)
        s["freq"] = freq.cuda()
        # the library's form of a frequency: 2^64 ths of a turn per position
        turns = [round(float(f) / TWO_PI * 2.0 ** 64) % 2 ** 64 for f in freq]
        s["steps"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64).cuda()
        s["query"], s["key"] = randn(T, H * D), randn(T, Hk * D)
        s["query_out"] = torch.empty_like(s["query"])
        if case["paged"]:
            s["value"] = randn(T, Hk * D)
            s["key_cache"], s["value_cache"] = (randn(blocks, case["block_size"], Hk, D) for _ in range(2))
        else:
            s["key_out"] = torch.empty_like(s["key"])
    else:
        H = case["heads"]
        s["key_cache"], s["value_cache"] = (randn(blocks, case["block_size"], Hk, D) for _ in range(2))
        s["query"] = randn(T, H * D, std=1.5)
        s["positions"] = s["past"][s["owner"]] + depth.cuda()
        words = -(-case["draft"] // 32)
        masks = []
        for par in plan["parents"]:
            rows = []
            for j, p in enumerate(par):
                rows.append((rows[p] if p >= 0 else 0) | 1 << j)
            masks += [[(m >> 32 * w) & 0xFFFFFFFF for w in range(words)] for m in rows]
        mask = torch.tensor(masks, dtype=torch.int64)
        s["mask"] = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32).cuda()
        s["slopes"] = s["sink"] = None
        if case["bias"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H).float()
        if case["sink"]:
            s["sink"] = randn(H, std=2.0)
        s["out"] = torch.empty_like(s["query"])
    if own:
        _handles(case, s)
    return s


def _handles(case, s):
    """What a program of this library keeps next to its tensors: the layer's handle."""
    import paged_kv_cache_reshape_gb300 as pa
    s["pa"] = pa
    if case["kind"] == "rotary":
        s["rotary"] = pa.make_rotary_config(case["head_size"], rotary_dim=case["rotary_dim"],
                                            rotary_offset=case["rotary_offset"],
                                            interleaved=int(case["interleaved"]),
                                            dtype=dict(fp16=pa.PA_ROTARY_FP16, bf16=pa.PA_ROTARY_BF16,
                                                       fp32=pa.PA_ROTARY_FP32)[case["dtype"]],
                                            attention_factor=s["factor"])
        if not case["paged"]:
            return
    pool = s["pools"][0, 0] if case["kind"] == "commit" else s["key_cache"]
    cfg = pa.make_config(case.get("heads", case["kv_heads"]), case["kv_heads"], case["head_size"],
                         case["block_size"], pool.shape[0], s["table"].shape[1], case["batch"], s["T"],
                         softcap=case.get("softcap", 0.0), local_window_size=case.get("window", -1),
                         cache_dtype=pa.PA_CACHE_BF16 if case["dtype"] == "bf16" else pa.PA_CACHE_FP16)
    s["tree"] = pa.PagedTree(cfg, case["draft"])
    if case["kind"] == "commit":
        s["layers"] = pa.layer_pools([p[0] for p in s["pools"]], [p[1] for p in s["pools"]])


def run(s):
    return {"rotary": _rotary, "tree": _tree, "commit": _commit}[s["case"]["kind"]](s)


def _rotary(s):
    case = s["case"]
    if own:
        pa, T = s["pa"], s["T"]
        if case["paged"]:
            s["tree"].write(s["rotary"], s["steps"], s["positions"], s["query"], s["key"], s["value"],
                            s["query_out"], s["key_cache"], s["value_cache"], s["table"], s["cum"], s["past"],
                            case["batch"], T)
            return [s["query_out"], s["key_cache"], s["value_cache"]]
        pa.pa_rotary(s["rotary"], s["steps"], s["positions"], T, case["heads"], s["query"], s["query_out"],
                     case["kv_heads"], s["key"], s["key_out"])
        return [s["query_out"], s["key_out"]]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None, :] for f in (torch.cos, torch.sin))

    def rotate(rows, heads):
        R, at = case["rotary_dim"], case["rotary_offset"]
        x = rows.view(rows.shape[0], heads, case["head_size"]).float()
        y = x.clone()
        part = x[..., at:at + R]
        if case["interleaved"]:
            x1, x2 = part[..., 0::2], part[..., 1::2]
            y[..., at:at + R:2], y[..., at + 1:at + R:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        else:
            x1, x2 = part[..., :R // 2], part[..., R // 2:]
            y[..., at:at + R // 2], y[..., at + R // 2:at + R] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        return y.to(rows.dtype).view_as(rows)

    query, key = rotate(s["query"], case["heads"]), rotate(s["key"], case["kv_heads"])
    if not case["paged"]:
        return [query, key]
    bs = case["block_size"]
    at = (s["past"][s["owner"]] + torch.arange(s["T"], device="cuda") - s["cum"][s["owner"]]).long()
    slot = s["table"][s["owner"], at // bs].long() * bs + at % bs
    s["key_cache"].view(-1, key.shape[1])[slot] = key
    s["value_cache"].view(-1, key.shape[1])[slot] = s["value"]
    return [query, s["key_cache"], s["value_cache"]]


def _tree(s):
    case = s["case"]
    if own:
        s["tree"].attention(s["query"], s["key_cache"], s["value_cache"], s["table"], s["cum"], s["past"],
                            case["batch"], s["T"], s["out"], positions=s["positions"], tree_mask=s["mask"],
                            distance_slopes=s["slopes"], head_sink=s["sink"])
        return s["out"]
    B, H, Hk, D, bs, n = (case[k] for k in ("batch", "heads", "kv_heads", "head_size", "block_size", "draft"))
    G, L = H // Hk, s["table"].shape[1] * bs
    pages = s["table"].clamp(min=0).long()
    K, V = (c[pages].view(B, L, Hk, D).permute(0, 2, 1, 3).float() for c in (s["key_cache"], s["value_cache"]))
    j = torch.arange(s["T"], device="cuda") - s["cum"][s["owner"]]
    q = torch.zeros(B, n, H, D, device="cuda")
    q[s["owner"], j] = s["query"].view(-1, H, D).float()
    q = q.view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    x = (q @ K.transpose(2, 3)).mul_(D ** -0.5)
    if case["softcap"]:
        x = torch.tanh_(x.div_(case["softcap"])).mul_(case["softcap"])
    x = x.view(B, Hk, n, G, L)
    # which key each row admits, and where it stands
    slot = torch.arange(L, device="cuda")
    node = slot - s["past"][:, None]
    bit = (s["mask"][:, :, None] >> torch.arange(32, device="cuda") & 1).flatten(1).bool()[:, :n]
    seen = torch.zeros(B, n, n, dtype=torch.bool, device="cuda")
    seen[s["owner"], j] = bit
    drafted = (node >= 0) & (node < s["n"][:, None])
    index = node.clamp(0, n - 1).long()
    seen = torch.gather(seen, 2, index[:, None, :].expand(B, n, L)) & drafted[:, None] | (node < 0)[:, None]
    qpos = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    qpos[s["owner"], j] = s["positions"]
    kpos = torch.where(drafted, torch.gather(qpos, 1, index), slot[None].int())
    if case["window"] > 0:
        seen &= kpos[:, None] > qpos[..., None] - case["window"]
    if s["slopes"] is not None:
        x += s["slopes"].view(1, Hk, 1, G, 1) * (kpos[:, None] - qpos[..., None]).float()[:, None, :, None]
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp_(x.sub_(top))
    den = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        den = den + torch.exp(s["sink"].float().view(1, Hk, 1, G, 1) - top)
    o = p.view(B, Hk, n * G, L) @ V / den.view(B, Hk, n * G, 1).clamp(min=torch.finfo(torch.float32).tiny)
    o = o.view(B, Hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H * D)
    return o[s["owner"], j].to(s["query"].dtype)


def _commit(s):
    case = s["case"]
    if own:
        s["tree"].commit(s["layers"], s["table"], s["past"], s["accepted"], s["count"], case["batch"],
                         new_past=s["new_past"])
        return [s["pools"], s["new_past"]]
    bs, most = case["block_size"], case["most"]
    rows = s["pools"].view(case["layers"], 2, -1, case["kv_heads"] * case["head_size"])
    i = torch.arange(most, device="cuda")
    b, i = torch.nonzero(i[None] < s["count"][:, None], as_tuple=True)

    def slots(at):
        at = (s["past"][b] + at).long()
        return s["table"][b, at // bs].long() * bs + at % bs

    rows[:, :, slots(i)] = rows[:, :, slots(s["accepted"][b, i])]
    return [s["pools"], s["past"] + s["count"]]


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    plan = _plan(case)
    bs, D, Hk = case["block_size"], case["head_size"], case["kv_heads"]
    if case["kind"] == "commit":
        pools = s["pools"].clone()
        flat = pools.view(case["layers"], 2, -1, Hk, D)
        before = s["pools"].view(case["layers"], 2, -1, Hk, D)
        table = s["table"].tolist()
        for b, path in enumerate(plan["paths"]):
            for i, a in enumerate(path):
                to, of = plan["past"][b] + i, plan["past"][b] + a
                flat[:, :, table[b][to // bs] * bs + to % bs] = before[:, :, table[b][of // bs] * bs + of % bs]
        return [pools, None]
    H, T = case["heads"], s["T"]
    if case["kind"] == "rotary":
        R, at = case["rotary_dim"], case["rotary_offset"]
        first, second = ((slice(at, at + R, 2), slice(at + 1, at + R, 2)) if case["interleaved"] else
                         (slice(at, at + R // 2), slice(at + R // 2, at + R)))
        z = torch.polar(torch.full((T, R // 2), float(s["factor"]), dtype=torch.float64, device="cuda"),
                        torch.outer(s["positions"].double(), s["freq"]))[:, None]
        out = []
        for rows, heads in ((s["query"], H), (s["key"], Hk)):
            x = rows.double().view(T, heads, D)
            w = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = w.real, w.imag
            out.append(x.reshape(T, heads * D))
        if not case["paged"]:
            return out
        pools = [s["key_cache"].double().view(-1, Hk * D), s["value_cache"].double().view(-1, Hk * D)]
        table, slot = s["table"].tolist(), []
        for b, n in enumerate(plan["n"]):
            slot += [table[b][p // bs] * bs + p % bs for p in range(plan["past"][b], plan["past"][b] + n)]
        slot = torch.tensor(slot, device="cuda")
        pools[0][slot], pools[1][slot] = out[1], s["value"].double()
        return [out[0]] + [p.view_as(s["key_cache"]) for p in pools]
    if work(case)["flops"] > 4e12:
        return None
    out, t = torch.zeros(T, H, D, dtype=torch.float64, device="cuda"), 0
    for b, (n, past) in enumerate(zip(plan["n"], plan["past"])):
        pages = s["table"][b, :-(-(past + n) // bs)].long()
        kv = [c[pages].reshape(-1, Hk, D)[:past + n] for c in (s["key_cache"], s["value_cache"])]
        dep = torch.tensor(plan["depths"][b], device="cuda")
        kpos = torch.cat([torch.arange(past, device="cuda"), past + dep])
        ok = torch.zeros(n, past + n, dtype=torch.bool, device="cuda")
        ok[:, :past] = True
        for j in range(n):
            a = j
            while a >= 0:
                ok[j, past + a] = True
                a = plan["parents"][b][a]
        gap = kpos[None, :] - (past + dep)[:, None]
        if case["window"] > 0:
            ok &= gap > -case["window"]
        for h in range(H):
            k, v = (c[:, h // (H // Hk)].double() for c in kv)
            x = s["query"].view(T, H, D)[t:t + n, h].double() @ k.T / math.sqrt(D)
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if s["slopes"] is not None:
                x = x + s["slopes"][h].double() * gap
            x = torch.where(ok, x, -math.inf)
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"][h].double().expand(n, 1)], 1)
            out[t:t + n, h] = torch.softmax(x, 1)[:, :past + n] @ v
        t += n
    return out.view(T, H * D)
