"""Cases of the tree-drafting operators, their plain form and their exact values.

Three operators of a speculative decode step over the compressed caches:

  norm_rope  RMSNorm of every query and key head with the position rotation
             (qk_norm_rope): of a prompt's tokens or of one token a sequence
  compress   the compressed entries that the drafted tokens of a tree complete
             (tree_compress), pooled along each node's own path
  attn       attention of every node of a tree of drafted tokens over the
             compressed cache, the drafted entries, the window and the sink
             (compressed_attn_tree), CSA (selected entries) and HCA (all)

A tree is parents[b, i] < i, the parent node of node i of sequence b (-1: the
node follows the last committed token, at position pos[b]; -2: no node).
Where ``own`` is false, run() computes them with elementary torch operations in
32 bits (rotation angles in 64) and rounds once at the end; where it is true,
it calls the package.
"""

import math

import torch

own = False

NONE = -2          # parents value of a place without a node


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # one new token of each of eight sequences, the decode step's query and row
        dict(name="norm_rope_decode", op="norm_rope", dtype="bf16", B=8, n=1, HQ=64, HK=1, d=512, r=64, fused=False, far=262144),
        # a prompt chunk of 16,384 tokens
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", B=1, n=16384, HQ=64, HK=1, d=512, r=64, fused=False, far=131072),
        # fp32, odd length, heads taken out of one fused projection (strided rows)
        dict(name="norm_rope_f32_fused", op="norm_rope", dtype="f32", B=3, n=2717, HQ=4, HK=1, d=64, r=16, fused=True, far=8192),
        # 64 drafted tokens of each of eight sequences, overlapped 4:1 entries
        dict(name="compress_csa", op="compress", kind="csa", dtype="bf16", B=8, T=64, m=4, c=512, r=64, norm=True, ctx=262144, tree="wide"),
        # the 128:1 entry that some paths complete
        dict(name="compress_hca", op="compress", kind="hca", dtype="bf16", B=8, T=32, m=128, c=512, r=64, norm=True, ctx=262142, tree="wide"),
        # the smallest useful tree: three drafted tokens in a row, one sequence
        dict(name="attn_csa_chain", op="attn", kind="csa", dtype="bf16", B=1, T=3, H=64, d=512, r=64, w=128, m=4, k=1024, ctx=16384, tree="chain", select=False),
        # a million-token context: selected entries of a gigabyte of cache
        dict(name="attn_csa_1m", op="attn", kind="csa", dtype="bf16", B=4, T=16, H=64, d=512, r=64, w=128, m=4, k=1024, ctx=1048576, tree="wide", select=False),
        # the same context through the 128:1 cache
        dict(name="attn_hca_1m", op="attn", kind="hca", dtype="bf16", B=4, T=16, H=64, d=512, r=64, w=128, m=128, k=0, ctx=1048576, tree="wide", select=False),
        # the widest trees: 512 nodes in one call
        dict(name="attn_hca_256k_wide", op="attn", kind="hca", dtype="bf16", B=8, T=64, H=64, d=512, r=64, w=128, m=128, k=0, ctx=262144, tree="wide", select=False),
        # the indexer selects inside the call, drafted entries among the candidates
        dict(name="attn_csa_select", op="attn", kind="csa", dtype="bf16", B=2, T=9, H=64, d=512, r=64, w=128, m=4, k=1024, ctx=65539, tree="wide", select=True, HI=64, dI=128),
        # fp32, small heads, odd tree
        dict(name="attn_csa_f32", op="attn", kind="csa", dtype="f32", B=3, T=7, H=4, d=64, r=16, w=16, m=4, k=16, ctx=509, tree="wide", select=False),
        # sixteen heads of 128 dims
        dict(name="attn_hca_16h", op="attn", kind="hca", dtype="bf16", B=2, T=11, H=16, d=128, r=64, w=128, m=128, k=0, ctx=8190, tree="wide", select=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "compress", "attn", "attn", "attn"])
    tree = rng.choice(["chain", "wide", "wide", "padded"])
    if op == "norm_rope":
        dtype, HQ, d, r = rng.choice([("bf16", 64, 512, 64), ("bf16", 16, 128, 64), ("f32", 4, 64, 16), ("f32", 64, 512, 64)])
        budget = 16384 * 64 * 512 // (HQ * d) // (2 if dtype == "f32" else 1)
        B = rng.randint(1, 8)
        return dict(op=op, dtype=dtype, B=B, n=_log(rng, 1, max(1, min(16384, budget) // B)), HQ=HQ, HK=1, d=d, r=r,
                    fused=rng.random() < 0.5, far=_log(rng, 32768, 1048576))
    if op == "compress":
        kind = rng.choice(["csa", "hca"])
        return dict(op=op, kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), B=rng.randint(1, 8), T=rng.randint(4, 64),
                    m=4 if kind == "csa" else 128, c=rng.choice([512, 512, 128]), r=64, norm=rng.random() < 0.7,
                    ctx=_log(rng, 300, 1048576) // 128 * 128 + (rng.randint(0, 127) if kind == "csa" else 127), tree=rng.choice(["chain", "wide", "padded"]))
    kind = rng.choice(["csa", "hca"])
    if rng.random() < 0.75:
        B = rng.randint(1, 8)
        T = _log(rng, 1, 64 if B <= 4 else 24)
        select = kind == "csa" and rng.random() < 0.25
        ctx = _log(rng, 200, 65536 if select else 262144)
        return dict(op=op, kind=kind, dtype="bf16", B=B if not select else min(B, 2), T=T if not select else min(T, 16), H=64, d=512, r=64, w=128,
                    m=4 if kind == "csa" else 128, k=rng.choice([1024, 1024, 517, 64]) if kind == "csa" else 0, ctx=ctx, tree=tree, select=select,
                    **(dict(HI=64, dI=128) if select else {}))
    dtype, H, d, r, w = rng.choice([("f32", 4, 64, 16, 16), ("bf16", 16, 128, 64, 128), ("f32", 3, 96, 32, 21)])
    return dict(op=op, kind=kind, dtype=dtype, B=rng.randint(1, 4), T=_log(rng, 1, 64), H=H, d=d, r=r, w=w,
                m=4 if kind == "csa" else 128, k=rng.choice([16, 64, 200]) if kind == "csa" else 0, ctx=_log(rng, 40, 8192), tree=tree, select=False)


def _keys_per_node(c):
    v = c["ctx"] // c["m"]
    return (min(c["k"], v) if c["kind"] == "csa" else v) + min(c["w"], c["ctx"])


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "norm_rope":
        rows = c["B"] * c["n"] * (c["HQ"] + c["HK"])
        return {"bytes": 2 * rows * c["d"] * e + 4 * c["B"] * c["n"], "flops": 6 * rows * c["d"]}
    if c["op"] == "compress":
        # per sequence: the nodes that complete an entry (one in m; for the 128:1 kind the sequences that stand at a block's end)
        S, R = (4, 2 * c["m"]) if c["kind"] == "csa" else (2, c["m"])
        rows = max(1, c["T"] // c["m"]) * c["B"]
        read = min(rows * R * 2, c["B"] * (R + c["T"]) * S)
        return {"bytes": (read + rows) * c["c"] * e, "flops": rows * R * c["c"] * 6}
    nodes, v = c["B"] * c["T"], c["ctx"] // c["m"]
    keys = _keys_per_node(c)
    # distinct cache rows of one sequence: all of them (HCA), or what T selections of k out of v cover
    rows = v if c["kind"] == "hca" else v * (1 - (1 - min(c["k"], v) / max(v, 1)) ** c["T"])
    bytes_ = c["B"] * (rows + min(c["w"], c["ctx"]) + c["T"]) * c["d"] * e + 2 * nodes * c["H"] * c["d"] * e
    flops = 4 * nodes * c["H"] * c["d"] * keys
    if c["select"]:
        bytes_ += c["B"] * v * c["dI"] * e + nodes * (c["HI"] * c["dI"] * e + 4 * c["k"])
        flops += 2 * nodes * v * c["HI"] * c["dI"]
    elif c["kind"] == "csa":
        bytes_ += 4 * nodes * c["k"]
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ inputs ----

def _tree(case, g):
    """parents [B][T] and pos [B] as host lists."""
    B, T, ctx, m = case["B"], case["T"], case["ctx"], case["m"]
    rnd = torch.rand(B, T + 2, generator=g).tolist()
    parents, pos = [], []
    for b in range(B):
        row = []
        live = T if case["tree"] != "padded" else max(1, int(T * (0.3 + 0.7 * rnd[b][T])))
        for i in range(T):
            if i >= live:
                row.append(NONE)
            elif case["tree"] == "chain" or i == 0:
                row.append(i - 1)
            else:                                    # one of the last few nodes; now and then another first token
                back = 1 + int(rnd[b][i] * 9)
                row.append(i - back if i - back >= 0 else (-1 if rnd[b][i] > 0.9 else 0))
        parents.append(row)
        # sequences stand at different lengths (the first one at ctx)
        back = 0 if b == 0 else int(rnd[b][T + 1] * min(ctx // 2, 777))
        pos.append(ctx - (back // m * m if case["op"] == "compress" else back))
    return parents, pos


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    gh = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    def gain(n):
        return 1.0 + 0.1 * torch.randn(n, generator=g, device=dev)

    s = {"case": c}
    if c["op"] == "norm_rope":
        B, n, HQ, HK, d = c["B"], c["n"], c["HQ"], c["HK"], c["d"]
        start = torch.randint(0, max(1, c["far"] - n), (B, 1), generator=gh)
        s["pos"] = (start + torch.arange(n)).to(torch.int32).to(dev)
        if c["fused"]:
            fused = normal(B, n, HQ + HK, d)
            s["q"], s["k"] = fused[:, :, :HQ], fused[:, :, HQ:]
        else:
            s["q"], s["k"] = normal(B, n, HQ, d), normal(B, n, HK, d)
        s["q_gain"], s["k_gain"] = gain(d), gain(d)
        return s
    B, T, m = c["B"], c["T"], c["m"]
    parents, pos = _tree(c, gh)
    s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
    if c["op"] == "compress":
        S, R, ch = (4, 2 * m, c["c"]) if c["kind"] == "csa" else (2, m, c["c"])
        s["ring"] = normal(B, R, S, ch)
        s["streams"] = tuple(normal(B, T, ch) for _ in range(S))
        s["bias_a"] = normal(m, ch, dtype=torch.float32, std=0.1)
        s["bias_b"] = normal(m, ch, dtype=torch.float32, std=0.1) if S == 4 else None
        s["gain"] = gain(ch) if c["norm"] else None
        s["out"] = torch.zeros(B, T, ch, dtype=dt, device=dev)
        return s
    H, d, w = c["H"], c["d"], c["w"]
    N = (c["ctx"] + T + 1) // m                      # room for every entry that the tree can complete
    s["q"] = normal(B, T, H, d)
    s["kv"] = normal(B, max(N, 1), d)
    s["win"] = normal(B, w, d)
    s["kv_raw"] = normal(B, T, d)
    s["draft"] = normal(B, T, d)
    s["sinks"] = torch.randn(H, generator=g, device=dev)
    s["q_gain"], s["kv_gain"] = gain(d), gain(d)
    s["out"] = torch.zeros(B, T, H, d, dtype=dt, device=dev)
    if c["select"]:
        # whole numbers: the scores are exact in any order of their sums, ties and all
        def whole(lo, hi, *shape):
            return torch.randint(lo, hi + 1, shape, generator=g, device=dev).to(dt)
        HI, dI = c["HI"], c["dI"]
        s["qI"], s["kI"], s["draft_kI"] = whole(-4, 4, B, T, HI, dI), whole(-4, 4, B, N, dI), whole(-4, 4, B, T, dI)
        s["wI"] = torch.randint(-8, 9, (B, T, HI), generator=g, device=dev).float() / 8
        s["idx"] = torch.full((B, T, c["k"]), -1, dtype=torch.int32, device=dev)
    elif c["kind"] == "csa":
        # k spread-out committed entries a node, its own drafted entries last
        k = c["k"]
        idx = torch.full((B, T, k), -1, dtype=torch.int64)
        u = torch.rand(B, T, k, generator=gh)
        for b in range(B):
            v = min(N, pos[b] // m)
            if v >= k:
                idx[b] = ((torch.arange(k) + u[b].double()) * v / k).long().clamp(max=v - 1)
            else:
                idx[b, :, :v] = torch.arange(v)
            depth = []
            for i, p in enumerate(parents[b]):
                depth.append(-1 if p == NONE else (depth[p] + 1 if p >= 0 else 0))
                mine, j = [], i
                while p != NONE and j >= 0:
                    if (pos[b] + depth[j] + 1) % m == 0:
                        mine.append(N + j)
                    j = parents[b][j]
                mine = mine[::-1][:k]
                at = min(v, k - len(mine))
                if mine:
                    idx[b, i, at:at + len(mine)] = torch.tensor(mine)
        s["idx"] = idx.to(torch.int32).to(dev)
    return s


# ---------------------------------------------------------------- plain form ----

def _rope(x, pos, r, sign=1.0):
    """x [..., d] with pos broadcast over x's leading dims: pairs (2j, 2j+1) of the last r dims."""
    d = x.shape[-1]
    j = torch.arange(r // 2, device=x.device, dtype=torch.float64)
    a = sign * pos.double()[..., None] * 10000.0 ** (-2.0 * j / r)
    cs, sn = a.cos().float(), a.sin().float()
    x0, x1 = x[..., d - r::2], x[..., d - r + 1::2]
    rot = torch.stack([x0 * cs - x1 * sn, x0 * sn + x1 * cs], dim=-1).flatten(-2)
    return torch.cat([x[..., :d - r], rot], dim=-1)


def _norm(x, gain):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain


def _plan(parents):
    """on[b, i, j]: node j is node i or an ancestor of it; depth [B, T]."""
    B, T = parents.shape
    live = parents >= -1
    on = torch.eye(T, device=parents.device).expand(B, T, T) * live[..., None]
    jump = (parents[..., None] == torch.arange(T, device=parents.device)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        on = ((on + jump @ on) > 0).float()
        jump = jump @ jump
    on = on > 0
    return on, on.sum(-1) - 1, live


def _plain_norm_rope(s):
    c = s["case"]
    q, k = _norm(s["q"].float(), s["q_gain"]), _norm(s["k"].float(), s["k_gain"])
    pos = s["pos"][..., None]
    return _rope(q, pos, c["r"]).to(s["q"].dtype), _rope(k, pos, c["r"]).to(s["k"].dtype)


def _plain_compress(s):
    c = s["case"]
    B, T, m = c["B"], c["T"], c["m"]
    csa = c["kind"] == "csa"
    R = 2 * m if csa else m
    on, depth, live = _plan(s["parents"])
    t = s["pos"][:, None] + depth
    done = live & ((t + 1) % m == 0)
    first = (t + 1) // m * m - m                      # first token of the completed block
    toks = first[..., None] + torch.arange(-m if csa else 0, m, device=t.device)           # [B, T, R]
    # the node on the path at each drafted position
    want = toks - s["pos"][:, None, None]
    at = (on[:, :, None, :] & (depth[:, None, None, :] == want[..., None])).float().argmax(-1)
    rows = []
    bi = torch.arange(B, device=t.device)[:, None, None]
    for j, x in enumerate(s["streams"]):
        ring = s["ring"][bi, toks % R, j].float()                                             # [B, T, R, c]
        rows.append(torch.where((want >= 0)[..., None], x[bi, at].float(), ring))
    if csa:
        a, b, za, zb = rows
        val = torch.cat([b[:, :, :m], a[:, :, m:]], 2)
        lb = (zb[:, :, :m] + s["bias_b"]).masked_fill((first <= 0)[..., None, None], float("-inf"))
        z = torch.cat([lb, za[:, :, m:] + s["bias_a"]], 2)
    else:
        val, z = rows[0], rows[1] + s["bias_a"]
    e = (z - z.amax(2, keepdim=True)).exp()
    y = (e * val).sum(2) / e.sum(2)
    if c["norm"]:
        y = _rope(_norm(y, s["gain"]), first, c["r"])
    return torch.where(done[..., None], y, torch.zeros_like(y)).to(s["out"].dtype)


def _plain_attn(s):
    c = s["case"]
    B, T, H, d, w, m, r = (c[x] for x in ("B", "T", "H", "d", "w", "m", "r"))
    on, depth, live = _plan(s["parents"])
    t = s["pos"][:, None] + depth
    N = s["kv"].shape[1]
    q = _rope(_norm(s["q"].float(), s["q_gain"]), t[..., None], r) * d ** -0.5
    rows = _rope(_norm(s["kv_raw"].float(), s["kv_gain"]), t, r)
    drafted = (t + 1) % m == 0
    drafted = drafted & ((t + 1) // m - 1 < N) & live
    idx = s.get("idx")
    if c["select"]:
        dots = torch.einsum("bthd,bnd->bthn", s["qI"].float(), torch.cat([s["kI"], s["draft_kI"]], 1).float())
        score = torch.einsum("bthn,bth->btn", dots.clamp(min=0), s["wI"])
        del dots
        seen = torch.arange(N, device=t.device) < (s["pos"] // m)[:, None]
        seen = torch.cat([seen[:, None].expand(B, T, N), on & drafted[:, None]], -1) & live[..., None]
        order = score.masked_fill(~seen, float("-inf")).sort(dim=-1, descending=True, stable=True).indices[..., :c["k"]]
        picked = torch.where(seen.gather(-1, order), order, torch.full_like(order, 1 << 30)).sort(-1).values
        picked = torch.where(picked == 1 << 30, torch.full_like(picked, -1), picked)
        idx = torch.nn.functional.pad(picked, (0, c["k"] - picked.shape[-1]), value=-1).to(torch.int32)
    out = torch.zeros_like(s["out"])
    for b in range(B):
        pos = s["pos"][b]
        slot = torch.arange(w, device=t.device)
        held = pos - 1 - (pos - 1 - slot) % w                                                  # position in ring slot
        see_ring = (held >= 0) & (held >= (t[b] - w + 1)[:, None])                             # [T, w]
        see_tree = on[b] & (t[b][None] >= (t[b] - w + 1)[:, None])                             # [T, T]
        near = torch.cat([s["win"][b].float(), rows[b]])
        see = torch.cat([see_ring, see_tree], 1)
        ln = (q[b].reshape(T * H, d) @ near.T).view(T, H, -1).masked_fill(~see[:, None], float("-inf"))
        if c["kind"] == "hca":
            v = torch.arange(N, device=t.device) < pos // m
            far = torch.cat([s["kv"][b].float(), s["draft"][b].float()])
            see_far = torch.cat([v.expand(T, N), on[b] & drafted[b]], 1)
            lf = (q[b].reshape(T * H, d) @ far.T).view(T, H, -1).masked_fill(~see_far[:, None], float("-inf"))
        else:
            at = idx[b].long()                                                                 # [T, k]
            far = s["kv"][b][at.clamp(0, N - 1)]
            far = torch.where((at >= N)[..., None], s["draft"][b][(at - N).clamp(0, T - 1)], far).float()
            lf = (q[b] @ far.transpose(1, 2)).masked_fill((idx[b] < 0)[:, None], float("-inf"))
        z = s["sinks"][None, :, None]
        mx = torch.maximum(torch.maximum(lf.amax(-1, keepdim=True), ln.amax(-1, keepdim=True)), z)
        ef, en = (lf - mx).exp(), (ln - mx).exp()
        den = ef.sum(-1, keepdim=True) + en.sum(-1, keepdim=True) + (z - mx).exp()
        of = (ef.reshape(T * H, -1) @ far).view(T, H, d) if c["kind"] == "hca" else ef @ far
        o = (of + (en.reshape(T * H, -1) @ near).view(T, H, d)) / den
        o = _rope(o, t[b][:, None], r, -1.0)
        out[b] = torch.where(live[b][:, None, None], o, torch.zeros_like(o)).to(out.dtype)
    return (out, idx) if c["select"] else out


# ----------------------------------------------------------------------- run ----

def run(s):
    c = s["case"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "compress": _plain_compress, "attn": _plain_attn}[c["op"]](s)
    from long_context_compressed_overlapped_b200 import api
    if c["op"] == "norm_rope":
        return api.qk_norm_rope(s["q"], s["k"], s["pos"], rope_dims=c["r"], q_gain=s["q_gain"], k_gain=s["k_gain"])
    if c["op"] == "compress":
        return api.tree_compress(c["kind"], s["streams"], s["ring"], s["pos"], s["parents"], s["bias_a"], c["m"], bias_b=s["bias_b"],
                                 gain=s["gain"], rms_norm=c["norm"], rope_dims=c["r"] if c["norm"] else 0, out=s["out"])
    kw = {}
    if c["select"]:
        kw = dict(k=c["k"], qI=s["qI"], wI=s["wI"], kI=s["kI"], draft_kI=s["draft_kI"], idx_out=s["idx"])
    elif c["kind"] == "csa":
        kw = dict(idx_in=s["idx"])
    out = api.compressed_attn_tree(c["kind"], s["q"], s["pos"], s["parents"], s["kv"], s["win"], s["kv_raw"], s["sinks"], m=c["m"],
                                   rope_dims=c["r"], draft=s["draft"], q_gain=s["q_gain"], kv_gain=s["kv_gain"], out=s["out"], **kw)
    return (out, s["idx"]) if c["select"] else out


# --------------------------------------------------------------------- exact ----

def _turn(x, pos, r):
    """Rotation as a complex product, 64 bits: x [..., d], pos a tensor over x's leading dims."""
    keep, rot = x[..., :x.shape[-1] - r], x[..., x.shape[-1] - r:]
    z = torch.view_as_complex(rot.reshape(*rot.shape[:-1], r // 2, 2).contiguous())
    freq = torch.exp(-torch.arange(0, r, 2, device=x.device, dtype=torch.float64) / r * math.log(10000.0))
    z = z * torch.polar(torch.ones_like(freq), torch.as_tensor(pos, dtype=torch.float64, device=x.device)[..., None] * freq)
    return torch.cat([keep, torch.view_as_real(z).flatten(-2)], -1)


def _unit(x, gain):
    return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * gain.double()


def _path(parents, i):
    """Nodes from the first drafted token down to node i."""
    up = []
    while i >= 0:
        up.append(i)
        i = parents[i]
    return up[::-1]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm_rope":
        got = []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            parts = [_turn(_unit(x[:, i:i + 2048].double(), gain), s["pos"][:, i:i + 2048, None], c["r"]) for i in range(0, x.shape[1], 2048)]
            got.append(torch.cat(parts, 1))
        return tuple(got)
    parents, pos, m = s["parents"].tolist(), s["pos"].tolist(), c["m"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    if c["op"] == "compress":
        R = s["ring"].shape[1]
        for b in range(c["B"]):
            for i in range(c["T"]):
                if parents[b][i] == NONE:
                    continue
                path = _path(parents[b], i)
                t = pos[b] + len(path) - 1
                if (t + 1) % m:
                    continue

                def token(p, j):
                    return (s["streams"][j][b, path[p - pos[b]]] if p >= pos[b] else s["ring"][b, p % R, j]).double()
                vals, logits = [], []
                for o in range(m):
                    p = t - m + 1 + o
                    vals.append(token(p, 0))
                    logits.append(token(p, 2 if c["kind"] == "csa" else 1) + s["bias_a"][o].double())
                    if c["kind"] == "csa" and t + 1 > m:
                        vals.append(token(p - m, 1))
                        logits.append(token(p - m, 3) + s["bias_b"][o].double())
                y = (torch.softmax(torch.stack(logits), 0) * torch.stack(vals)).sum(0)
                out[b, i] = _turn(_unit(y, s["gain"]), t + 1 - m, c["r"]) if c["norm"] else y
        return out
    w, d, r, N = c["w"], c["d"], c["r"], s["kv"].shape[1]
    picked = s["idx"].clone().long() if c["kind"] == "csa" else None
    for b in range(c["B"]):
        for i in range(c["T"]):
            if parents[b][i] == NONE:
                continue
            path = _path(parents[b], i)
            t = pos[b] + len(path) - 1
            new = [j for n, j in enumerate(path) if (pos[b] + n + 1) % m == 0 and (pos[b] + n + 1) // m - 1 < N]
            v = min(N, pos[b] // m)
            if c["select"]:
                key = torch.cat([s["kI"][b, :v], s["draft_kI"][b, new]]).double()
                name = torch.tensor(list(range(v)) + [N + j for j in new], device=key.device)
                score = (s["wI"][b, i].double()[:, None] * (s["qI"][b, i].double() @ key.T).clamp(min=0)).sum(0)
                best = name[torch.sort(-score, stable=True).indices[:c["k"]]].sort().values
                picked[b, i] = -1
                picked[b, i, :len(best)] = best
            if c["kind"] == "csa":
                sel = picked[b, i][picked[b, i] >= 0]
                far = torch.cat([s["kv"][b, sel[sel < N]], s["draft"][b, sel[sel >= N] - N]])
            else:
                far = torch.cat([s["kv"][b, :v], s["draft"][b, new]])
            old = [p for p in range(max(0, t - w + 1), pos[b])]
            ring = s["win"][b, [p % w for p in old]].double()
            fresh = [(n, j) for n, j in enumerate(path) if pos[b] + n > t - w]
            rows = _turn(_unit(s["kv_raw"][b, [j for _, j in fresh]].double(), s["kv_gain"]),
                         torch.tensor([pos[b] + n for n, _ in fresh]), r)
            keys = torch.cat([far.double(), ring, rows])
            q = _turn(_unit(s["q"][b, i].double(), s["q_gain"]), torch.full((c["H"],), t), r)
            logit = torch.cat([q @ keys.T / math.sqrt(d), s["sinks"].double()[:, None]], 1)
            o = torch.softmax(logit, 1)[:, :-1] @ keys
            out[b, i] = _turn(o, torch.full((c["H"],), -t), r)
    return (out, picked.to(torch.int32)) if c["select"] else out
