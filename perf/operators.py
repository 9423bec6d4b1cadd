"""Cases that time and compare the serving operators around the paged tree verification.

Four operators: `plan` builds block tables and slot maps from request lengths, `store` writes new
K/V rows into the paged pools, `diff` is differential attention of draft trees over a cache, and
`w4` multiplies activations with 4-bit weights.  `own = False` computes them in plain torch
operations; `own = True` calls this package's kernels on the same state.
"""
import math

import numpy as np
import torch

own = False

HEAD = 128                                  # dims of a head: two maps of 64 in `diff`


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One request's 64-node tree: the latency of planning a single stream's step.
        dict(name="plan_one_tree", op="plan", B=1, page=16, kv_lo=4096, kv_hi=4096, new_lo=64,
             new_hi=64, short=False),
        # 512 running requests with 4-node chains, some of them finished and giving pages back.
        dict(name="plan_512_chains", op="plan", B=512, page=16, kv_lo=512, kv_hi=4096, new_lo=4,
             new_hi=4, short=False),
        # 64 prompts admitted at once, ragged, one token among them.
        dict(name="plan_64_prompts", op="plan", B=64, page=64, kv_lo=0, kv_hi=0, new_lo=1,
             new_hi=8192, short=False),
        # The K/V rows of a 16-node tree on 8 KV heads: a store's latency.
        dict(name="store_tree", op="store", n=16, hkv=8, page=16),
        # A long prompt's rows, read in place out of a fused projection, with padding behind them.
        dict(name="store_prompt", op="store", n=32749, hkv=8, page=64),
        # One request, 64-node tree, 4K cache, the 27B shape.
        dict(name="diff_one_4k", op="diff", B=1, n=64, kv_lo=4096, kv_hi=4096, hq=40, hkv=8,
             page=0, norm=True),
        # 33 requests decoding one token each over 16-token pages, a small head layout.
        dict(name="diff_decode_33", op="diff", B=33, n=1, kv_lo=1, kv_hi=2000, hq=8, hkv=2,
             page=16, norm=False),
        # 64 requests with 16-node trees over ragged paged caches.
        dict(name="diff_64_paged", op="diff", B=64, n=16, kv_lo=1024, kv_hi=8192, hq=40, hkv=8,
             page=64, norm=True),
        # One request with a 128K cache.
        dict(name="diff_one_128k", op="diff", B=1, n=16, kv_lo=131072, kv_hi=131072, hq=40, hkv=8,
             page=0, norm=True),
        # A single token through a square projection: the smallest product of a decode step.
        dict(name="w4_one_row", op="w4", M=1, N=5120, K=5120, group=128, zeros=False, f32=False),
        # The fused q/k/v projection of a 16-node tree, with zero points and finer groups.
        dict(name="w4_qkv_16", op="w4", M=16, N=7168, K=5120, group=64, zeros=True, f32=False),
        # The vocabulary projection of a 64-node tree, logits in 32 bits.
        dict(name="w4_head_64", op="w4", M=64, N=151936, K=5120, group=128, zeros=True, f32=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "diff", "diff", "w4", "w4"])
    if op == "plan":
        page = rng.choice([16, 32, 64, 128, 256])
        if rng.random() < 0.5:              # trees over running requests
            hi = _log_int(rng, 64, 16384)
            return dict(op="plan", B=_log_int(rng, 1, 2048), page=page, kv_lo=rng.randint(0, hi),
                        kv_hi=hi, new_lo=1, new_hi=rng.randint(1, 64),
                        short=rng.random() < 0.2)
        hi = _log_int(rng, 16, 65536)       # prompts
        return dict(op="plan", B=max(1, min(_log_int(rng, 1, 256), 500000 // hi)), page=page,
                    kv_lo=0, kv_hi=rng.choice([0, 777]), new_lo=1, new_hi=hi,
                    short=rng.random() < 0.2)
    if op == "store":
        return dict(op="store", n=_log_int(rng, 1, 32749), hkv=rng.randint(1, 8),
                    page=rng.choice([16, 32, 64, 128]))
    if op == "diff":
        hkv = rng.choice([1, 2, 4, 8])
        G = rng.randint(1, 8)
        B, n = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 131072)
        hi = max(1, min(hi, 64 * 16 * 40 * 8192 // (B * n * hkv * G), 64 * 8192 * 8 // (B * hkv)))
        return dict(op="diff", B=B, n=n, kv_lo=rng.randint(0, hi), kv_hi=hi, hq=hkv * G, hkv=hkv,
                    page=rng.choice([0, 16, 32, 64, 128]), norm=rng.random() < 0.7)
    group = rng.choice([32, 64, 128])
    M, K = _log_int(rng, 1, 96), group * max(1, _log_int(rng, 256, 8192) // group)
    return dict(op="w4", M=M, N=max(1, min(_log_int(rng, 64, 40000), 64 * 151936 * 5120 // (M * K))),
                K=K, group=group, zeros=rng.random() < 0.5, f32=rng.random() < 0.3)


# ------------------------------------------------------------------------------------ the inputs
def _lengths(B, lo, hi):
    """B lengths spread over [lo, hi], both ends among them: the case's own, whatever the seed."""
    return np.linspace(hi, lo, B).round().astype(np.int64)


def _requests(c):
    """A plan's requests, before the seed shuffles them: cached and new tokens, pages held."""
    rs, B, P = np.random.RandomState(17), c["B"], c["page"]
    kv = rs.permutation(_lengths(B, c["kv_lo"], c["kv_hi"]))
    new = rs.permutation(_lengths(B, c["new_lo"], c["new_hi"]))
    held = (kv + P - 1) // P                # what the cache needs now
    if B >= 8:
        over = rs.rand(B) < 0.25            # reserved for a tree of which little was accepted
        held = held + over * rs.randint(0, 64 // P + 2, size=B)
        done = (rs.rand(B) < 0.05) & (c["kv_hi"] > 0)   # finished: gives everything back
        kv, new = np.where(done, 0, kv), np.where(done, 0, new)
    return kv, new, held


def _nodes(c):
    """A batch's cached tokens and tree sizes, before the seed shuffles them."""
    rs = np.random.RandomState(19)
    return (_lengths(c["B"], c["kv_lo"], c["kv_hi"]),
            rs.permutation(_lengths(c["B"], (c["n"] + 1) // 2, c["n"])))


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) + 1)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", dtype=torch.float32, generator=g).to(torch.bfloat16)


def _starts(x):
    cu = np.zeros(len(x) + 1, np.int32)
    np.cumsum(x, out=cu[1:])
    return cu


def _prepare_plan(c, seed):
    rs = np.random.RandomState((int(seed) * 7919 + 11) % (1 << 31))
    order = rs.permutation(c["B"])
    kv, new, held = (x[order].astype(np.int32) for x in _requests(c))
    cu = _starts(new)
    P, used = c["page"], int(held.sum())
    max_pages = (c["kv_hi"] + c["new_hi"] + P - 1) // P + 64 // P + 2
    num_pages = c["B"] * max_pages + 64
    if c["short"]:                          # a pool with pages for half of what is asked for
        grow = np.maximum(0, (kv + new + P - 1) // P - held)
        num_pages = used + int(grow.sum()) // 2 + 1
    pages = rs.permutation(num_pages).astype(np.int32)
    bt = np.full((c["B"], max_pages), -1, np.int32)
    bt[np.arange(max_pages)[None, :] < held[:, None]] = pages[:used]
    ring = np.zeros(num_pages, np.int32)    # the free list is a ring: [head, tail) modulo its size
    head = int(rs.randint(0, num_pages))
    ring[(head + np.arange(num_pages - used)) % num_pages] = pages[used:]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(case=c, cu_new=_dev(cu), kv_len=_dev(kv), held=_dev(held), ring=_dev(ring),
                ring_state=_dev(np.array([head, head + num_pages - used], np.int64)),
                block_table=_dev(bt), num_pages=num_pages,
                held_out=torch.empty(c["B"], **i32), slot_cap=torch.empty(c["B"], **i32),
                state_out=torch.empty(2, dtype=torch.int64, device="cuda"),
                slot_map=torch.empty(int(cu[-1]) + 5, dtype=torch.int64, device="cuda"),
                ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))


def _prepare_store(c, seed):
    g = _gen(seed)
    n, hkv, P = c["n"], c["hkv"], c["page"]
    pad = 3                                 # rows behind the last token, of a padded batch
    fused = _normal(g, n + pad, 2 * hkv * HEAD)
    num_pages = (n + P - 1) // P + 3
    slots = torch.randperm(num_pages, device="cuda", generator=g)[:, None] * P
    slots = (slots + torch.arange(P, device="cuda")).reshape(-1)[:n + pad].contiguous()
    slots[n:] = -1
    pools = [_normal(g, num_pages * P, hkv, HEAD) for _ in range(2)]
    return dict(case=c, k=fused[:, :hkv * HEAD].unflatten(1, (hkv, HEAD)),
                v=fused[:, hkv * HEAD:].unflatten(1, (hkv, HEAD)), slots=slots, k_pool=pools[0],
                v_pool=pools[1], ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))


def _prepare_diff(c, seed):
    rs = np.random.RandomState((int(seed) * 104729 + 3) % (1 << 31))
    g = _gen(seed)
    B, hq, hkv, P = c["B"], c["hq"], c["hkv"], c["page"]
    order = rs.permutation(B)
    kv, nodes = (x[order].astype(np.int32) for x in _nodes(c))
    cu = _starts(nodes)
    local = np.concatenate([np.arange(m) for m in nodes])
    back = (rs.rand(local.size) ** 2 * np.minimum(local, 8)).astype(np.int64)
    parent = np.where(local == 0, -1, local - 1 - back).astype(np.int32)
    if P:
        max_pages = (int(kv.max()) + c["n"] + P - 1) // P
        num_pages = B * max_pages + 1
        table = rs.permutation(num_pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        slots = num_pages * P
    else:
        table, num_pages = np.zeros((1, 1), np.int32), 0
        slots = int(kv.sum()) + B * 7 + 64
    base = np.zeros(B, np.int64)
    base[1:] = np.cumsum(kv[:-1] + 7)
    nt = int(cu[-1])
    s = dict(case=c, cu=_dev(cu), parent=_dev(parent), tokens=_dev(np.zeros(nt, np.int32)),
             kv_len=_dev(kv), slot_base=_dev(base), kv_max=int(kv.max()), table=_dev(table),
             slot_cap=_dev((kv + 64).astype(np.int32)), q=_normal(g, nt, hq, HEAD),
             k_tree=_normal(g, nt, hkv, HEAD), v_tree=_normal(g, nt, hkv, HEAD),
             k_cache=_normal(g, slots, hkv, HEAD), v_cache=_normal(g, slots, hkv, HEAD),
             lam=torch.rand(hq, device="cuda", generator=g) * 0.6 + 0.2,
             norm_w=(1 + 0.1 * torch.randn(HEAD, device="cuda", generator=g)).to(torch.bfloat16)
             if c["norm"] else None, out_scale=0.2 if c["norm"] else 1.0,
             out=torch.empty(nt, hq, HEAD, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(nt, hq, 2, dtype=torch.float32, device="cuda"), keep={})
    return s


def _prepare_w4(c, seed):
    g = _gen(seed)
    M, N, K, group = c["M"], c["N"], c["K"], c["group"]
    scales = torch.randn(N, K // group, device="cuda", generator=g)
    return dict(case=c, x=_normal(g, M, K),
                wq=torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda",
                                 generator=g),
                scales=(0.005 * torch.exp(0.3 * scales)).to(torch.bfloat16),
                zeros=torch.randint(4, 12, (N, K // group), dtype=torch.uint8, device="cuda",
                                    generator=g) if c["zeros"] else None,
                out=torch.empty(M, N, dtype=torch.float32 if c["f32"] else torch.bfloat16,
                                device="cuda"), keep={})


def prepare(case, seed):
    return {"plan": _prepare_plan, "store": _prepare_store, "diff": _prepare_diff,
            "w4": _prepare_w4}[case["op"]](case, seed)


# ------------------------------------------------------------------------------- the plain forms
def _plain_plan(s):
    P, cap = s["case"]["page"], s["num_pages"]
    cu, kv, held = s["cu_new"].long(), s["kv_len"].long(), s["held"].long()
    need = (kv + cu[1:] - cu[:-1] + P - 1) // P
    grow, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    head, tail = s["ring_state"][0], s["ring_state"][1]
    upto = torch.cumsum(grow, 0)
    served = (grow == 0) | (upto <= tail - head)
    held_out = torch.where(served, need, held)
    bt = s["block_table"]
    col = torch.arange(bt.shape[1], device=bt.device)[None, :]
    fresh = (col >= held[:, None]) & (col < need[:, None]) & served[:, None]
    src = (head + (upto - grow)[:, None] + col - held[:, None]).remainder(cap)
    gone = (col >= need[:, None]) & (col < held[:, None])
    dst = (tail + (torch.cumsum(back, 0) - back)[:, None] + col - need[:, None]).remainder(cap)
    wide = torch.cat([s["ring"], s["ring"][:1]])       # one more place, for what is not given back
    wide.scatter_(0, torch.where(gone, dst, cap).reshape(-1), bt.reshape(-1))
    bt.copy_(torch.where(fresh, s["ring"][src], bt))
    s["ring"].copy_(wide[:cap])
    taken = torch.where(served, grow, 0).sum()
    tok = torch.arange(s["slot_map"].numel(), device=bt.device)
    r = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=held.numel() - 1)
    t = kv[r] + tok - cu[r]
    page = bt[r, (t // P).clamp(max=bt.shape[1] - 1)].long()
    ok = (tok < cu[-1]) & served[r]
    slot_map = torch.where(ok, page * P + t % P, -1)
    return dict(block_table=bt, held=held_out.int(), ring=s["ring"],
                state=torch.stack([head + taken, tail + back.sum()]),
                slot_cap=(held_out * P).int(), slot_map=slot_map)


def _plain_store(s):
    # every token's row goes to its slot; slots below zero are padding, and their rows rewrite
    # what the first token's slot gets anyway
    ok = (s["slots"] >= 0)[:, None, None]
    at = torch.where(s["slots"] >= 0, s["slots"], s["slots"][0])
    s["k_pool"][at] = torch.where(ok, s["k"], s["k"][:1])
    s["v_pool"][at] = torch.where(ok, s["v"], s["v"][:1])
    return dict(k_pool=s["k_pool"], v_pool=s["v_pool"])


def _plain_diff(s):
    c = s["case"]
    hq, hkv, P, n = c["hq"], c["hkv"], c["page"], c["n"]
    G = hq // hkv
    cu, L = s["cu"].long(), s["kv_len"].long()
    B, nt, Lm = c["B"], s["q"].shape[0], s["kv_max"]
    dev = cu.device
    tok = torch.arange(nt, device=dev)
    r = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    i = tok - cu[r]
    t = torch.arange(Lm, device=dev)[None, :].expand(B, Lm)
    inside = t < L[:, None]
    if P:
        at = torch.gather(s["table"].long(), 1, (t // P).contiguous()) * P + t % P
    else:
        at = s["slot_base"][:, None] + t
    at = torch.where(inside, at, 0)
    node = (cu[:-1, None] + torch.arange(n, device=dev)).clamp(max=nt - 1)

    def keys(cache, tree):                  # [B, hkv, keys, dims]: the cache, then the tree
        return torch.cat([cache[at], tree[node]], 1).float().transpose(1, 2)

    # who sees whom in a tree: ancestors are what (I + parent links) reaches in 63 steps
    link = torch.zeros(B, n, n, device=dev)
    up = s["parent"].long()
    link[r, i, up.clamp(min=0)] = (up >= 0).float()
    eye = torch.eye(n, device=dev)
    sees = torch.matrix_power(link + eye, 63) > 0
    mask = torch.cat([inside[:, None, :].expand(B, n, Lm), sees], 2)[:, None, None]
    q = torch.zeros(B, n, hq, HEAD, device=dev)
    q[r, i] = s["q"].float()
    q = q.view(B, n, hkv, G, 2, HEAD // 2).permute(0, 2, 4, 3, 1, 5)    # [B, hkv, map, G, n, 64]
    k = keys(s["k_cache"], s["k_tree"]).unflatten(3, (2, HEAD // 2)).transpose(2, 3)
    z = (q.flatten(3, 4) @ k.transpose(3, 4)).unflatten(3, (G, n)) * (HEAD // 2) ** -0.5
    z = torch.where(mask[:, :, None], z, -math.inf)
    top = z.amax(5, keepdim=True)
    e = torch.exp(z - top)
    sums = e.sum(5, keepdim=True)
    v = keys(s["v_cache"], s["v_tree"])
    o = ((e / sums).flatten(2, 4) @ v).unflatten(2, (2, G, n))          # [B, hkv, map, G, n, 128]
    lam = s["lam"].view(hkv, G, 1, 1)
    d = o[:, :, 0] - lam * o[:, :, 1]
    if s["norm_w"] is not None:
        d = d * torch.rsqrt(d.square().mean(-1, keepdim=True) + 1e-5) * s["norm_w"].float()
    d = (d * s["out_scale"]).permute(0, 3, 1, 2, 4).flatten(2, 3)       # [B, n, hq, 128]
    lse = (top + torch.log(sums))[..., 0].permute(0, 4, 1, 3, 2).flatten(2, 3)
    return dict(out=d[r, i].to(torch.bfloat16), lse=lse[r, i])


def _plain_w4(s):
    c = s["case"]
    N, K, group = c["N"], c["K"], c["group"]
    w = torch.stack([s["wq"] & 15, s["wq"] >> 4], 2).view(N, K // group, group).float()
    w -= 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w *= s["scales"].float()[..., None]
    return dict(out=(s["x"].float() @ w.view(N, K).t()).to(s["out"].dtype))


# ------------------------------------------------------------------------- the framework's calls
def _own_plan(s):
    from draft_tree_verification_masked_b200 import etree_page_plan
    etree_page_plan(s["cu_new"], s["kv_len"], s["case"]["page"], s["num_pages"], s["held"],
                    s["ring"], s["ring_state"], s["block_table"], s["held_out"], s["state_out"],
                    s["slot_cap"], s["slot_map"], s["ws"])
    return dict(block_table=s["block_table"], held=s["held_out"], ring=s["ring"],
                state=s["state_out"], slot_cap=s["slot_cap"], slot_map=s["slot_map"])


def _own_store(s):
    from draft_tree_verification_masked_b200 import etree_kv_store
    etree_kv_store(s["slots"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["ws"])
    return dict(k_pool=s["k_pool"], v_pool=s["v_pool"])


def _own_diff(s):
    import draft_tree_verification_masked_b200 as et
    c, keep = s["case"], s["keep"]
    if not keep:                            # the batch handle and workspace a program keeps
        keep["batch"] = et.make_batch(s["cu"], s["parent"], s["tokens"], s["kv_len"],
                                      s["slot_base"], s["slot_cap"], c["n"], s["kv_max"])
        keep["ws"] = torch.zeros(et.etree_attn_diff_workspace_size(keep["batch"], c["hq"],
                                                                   c["hkv"]),
                                 dtype=torch.uint8, device="cuda")
    args = (s["q"], s["k_tree"], s["v_tree"], s["k_cache"], s["v_cache"], (HEAD // 2) ** -0.5,
            s["lam"], s["norm_w"], 1e-5, s["out_scale"], s["out"], s["lse"], keep["ws"])
    if c["page"]:
        et.etree_verify_attn_diff_paged(keep["batch"], s["table"], c["page"], *args)
    else:
        et.etree_verify_attn_diff(keep["batch"], *args)
    return dict(out=s["out"], lse=s["lse"])


def _own_w4(s):
    import draft_tree_verification_masked_b200 as et
    c, keep = s["case"], s["keep"]
    if not keep:
        keep["ws"] = torch.zeros(et.etree_w4_workspace_size(c["M"], c["N"], c["K"]),
                                 dtype=torch.uint8, device="cuda")
    et.etree_w4_linear(s["x"], s["wq"], s["scales"], s["zeros"], c["group"], None, s["out"],
                       keep["ws"])
    return dict(out=s["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "store": _own_store, "diff": _own_diff, "w4": _own_w4}[op](state)
    return {"plan": _plain_plan, "store": _plain_store, "diff": _plain_diff,
            "w4": _plain_w4}[op](state)


# ------------------------------------------------------------------------------ what a pass needs
def work(case):
    c = case
    if c["op"] == "plan":
        P = c["page"]
        kv, new, held = _requests(c)
        need = (kv + new + P - 1) // P
        moved = np.abs(need - held).sum()   # pages taken and given back: an id read and written
        touched = np.where(new > 0, need - kv // P, 0).sum()    # table entries of the new tokens
        # per request two lengths and the pages held in, the pages held and the capacity out
        return dict(bytes=float(c["B"] * 5 * 4 + moved * 8 + touched * 4 + new.sum() * 8), flops=0)
    if c["op"] == "store":
        return dict(bytes=2 * 2 * c["n"] * c["hkv"] * HEAD * 2 + c["n"] * 8, flops=0)
    if c["op"] == "diff":
        kv, nodes = _nodes(c)
        per_node = 2 * c["hkv"] * HEAD * 2 + 2 * c["hq"] * HEAD * 2 + c["hq"] * 8
        # q k^T over 64 dims for each of two maps, and their products with 128-wide values
        pairs = nodes.mean() * kv.sum() + (nodes * nodes).sum()
        return dict(bytes=float(kv.sum() * 2 * c["hkv"] * HEAD * 2 + nodes.sum() * per_node),
                    flops=float(pairs * c["hq"] * (2 * 2 * 64 + 2 * 2 * HEAD)))
    M, N, K = c["M"], c["N"], c["K"]
    per_group = 3 if c["zeros"] else 2
    return dict(bytes=N * K / 2 + N * K / c["group"] * per_group + M * K * 2
                + M * N * (4 if c["f32"] else 2), flops=2 * M * N * K)


# ------------------------------------------------------------- the same outputs, in 64 bits, apart
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "plan":
        P, cap = c["page"], s["num_pages"]
        cu, kv, held = (s[k].tolist() for k in ("cu_new", "kv_len", "held"))
        bt, ring = s["block_table"].tolist(), s["ring"].tolist()
        head, tail = s["ring_state"].tolist()
        free, slots, after, back = tail - head, [], [], []
        stuck = False
        for r in range(c["B"]):
            need = -(-(kv[r] + cu[r + 1] - cu[r]) // P)
            grow = max(0, need - held[r])
            stuck = stuck or grow > free
            if grow and stuck:
                after.append(held[r])
                slots += [-1] * (cu[r + 1] - cu[r])
                continue
            back += bt[r][need:held[r]]
            for p in range(held[r], need):
                bt[r][p] = ring[head % cap]
                head, free = head + 1, free - 1
            after.append(need)
            slots += [bt[r][t // P] * P + t % P for t in range(kv[r], kv[r] + cu[r + 1] - cu[r])]
        for page in back:
            ring[tail % cap] = page
            tail += 1
        slots += [-1] * (s["slot_map"].numel() - len(slots))
        i32 = torch.int32
        return dict(block_table=torch.tensor(bt, dtype=i32), held=torch.tensor(after, dtype=i32),
                    ring=torch.tensor(ring, dtype=i32), state=torch.tensor([head, tail]),
                    slot_cap=torch.tensor([h * P for h in after], dtype=i32),
                    slot_map=torch.tensor(slots))
    if c["op"] == "store":
        keep = s["slots"] >= 0
        got = {}
        for name, rows in (("k_pool", s["k"]), ("v_pool", s["v"])):
            pool = s[name].double()
            pool.index_copy_(0, s["slots"][keep], rows[keep].double())
            got[name] = pool
        return got
    if c["op"] == "diff":
        hq, hkv = c["hq"], c["hkv"]
        cu, parent = s["cu"].tolist(), s["parent"].tolist()
        out = torch.zeros(cu[-1], hq, HEAD, dtype=torch.float64, device="cuda")
        lse = torch.zeros(cu[-1], hq, 2, dtype=torch.float64, device="cuda")
        for r in range(c["B"]):
            a, b, L = cu[r], cu[r + 1], int(s["kv_len"][r])
            pos = torch.arange(L, device="cuda")
            if c["page"]:
                rows = s["table"][r].long()[pos // c["page"]] * c["page"] + pos % c["page"]
            else:
                rows = pos + int(s["slot_base"][r])
            hidden = torch.ones(b - a, L + b - a, dtype=torch.bool)
            hidden[:, :L] = False
            for j in range(b - a):
                at = j
                while at >= 0:
                    hidden[j, L + at] = False
                    at = parent[a + at]
            hidden = hidden.cuda()
            for h in range(hkv):
                k = torch.cat([s["k_cache"][rows, h], s["k_tree"][a:b, h]]).double()
                v = torch.cat([s["v_cache"][rows, h], s["v_tree"][a:b, h]]).double()
                for qh in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                    q = s["q"][a:b, qh].double()
                    parts = []
                    for m in range(2):
                        cols = slice(64 * m, 64 * m + 64)
                        z = (q[:, cols] @ k[:, cols].T / 8.0).masked_fill(hidden, -math.inf)
                        lse[a:b, qh, m] = torch.logsumexp(z, 1)
                        parts.append(torch.softmax(z, 1) @ v)
                    out[a:b, qh] = parts[0] - s["lam"][qh].double() * parts[1]
        if s["norm_w"] is not None:
            out = out / (out.pow(2).mean(2, keepdim=True) + 1e-5).sqrt() * s["norm_w"].double()
        return dict(out=out * s["out_scale"], lse=lse)
    N, K, group = c["N"], c["K"], c["group"]
    x = s["x"].double()
    got = torch.empty(c["M"], N, dtype=torch.float64, device="cuda")
    for a in range(0, N, 16384):
        q = s["wq"][a:a + 16384]
        w = torch.empty(q.shape[0], K, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
        z = 8.0 if s["zeros"] is None else s["zeros"][a:a + 16384].double().repeat_interleave(group, 1)
        got[:, a:a + 16384] = x @ ((w - z)
                                   * s["scales"][a:a + 16384].double().repeat_interleave(group, 1)).T
    return dict(out=got)
