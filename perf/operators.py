"""The training read's gradients as cases: attention's backward pass under the prefix-shared layout, which
recomputes the probabilities from the forward's log-sum-exp, and the backward pass of the per-head norms with
their rotation.  `run` computes a case in its plain form (torch operations, 32 bits) or, with `own` set, by the
library's calls; `exact` is the definition in 64 bits."""
import math

import torch

own = False
EPS = 1e-6


def _read(name, n_q, n_kv, head_dim, window, blocks):
    return {"name": name, "op": "read_backward", "n_q": n_q, "n_kv": n_kv, "head_dim": head_dim, "window": window,
            "blocks": blocks}


def _prep(name, n_q, n_kv, head_dim, rope_dims, theta, k_eq_v, donor, kv_f32, blocks):
    return {"name": name, "op": "prep_backward", "n_q": n_q, "n_kv": n_kv, "head_dim": head_dim,
            "rope_dims": rope_dims, "theta": theta, "k_eq_v": k_eq_v, "donor": donor, "kv_f32": kv_f32,
            "blocks": blocks}


def listed():
    """`blocks`: rows of the shared prefix, then of each branch that continues it."""
    return [
        # a single short sequence: latency counts
        _read("read-short", 4, 2, 64, 0, "33"),
        # ragged branches, an empty one and a one-row one, a window that cuts into the prefix
        _read("read-ragged", 8, 2, 128, 100, "137,1,330,0,61,210"),
        # a sliding and a full layer of the 42-layer stack over its training pass
        _read("read-sliding", 8, 2, 256, 512, "1024,256,256,256,256"),
        _read("read-full", 16, 1, 512, 0, "1024,256,256,256,256"),
        # one long causal sequence with a kv head for each q head
        _read("read-causal", 8, 8, 128, 0, "4001"),
        # the full layer over a pass twice as long
        _read("read-full-long", 16, 1, 512, 0, "2048,1024,1024"),
        # a one-row pass: latency
        _prep("prep-one-row", 8, 2, 256, 256, 1e4, False, True, False, "1"),
        # a KV-sharing layer has no keys of its own; partial rotation, odd row count
        _prep("prep-sharer", 12, 4, 128, 64, 1e4, False, False, False, "500,277"),
        # the stack's sliding donor, and its full one (keys = values, partial rotation) whose key and value
        # gradients are the sums over the layers that read them
        _prep("prep-sliding", 8, 2, 256, 256, 1e4, False, True, False, "1024,256,256,256,256"),
        _prep("prep-full", 16, 1, 512, 128, 1e6, True, True, True, "1024,256,256,256,256"),
        # a long pass
        _prep("prep-long", 8, 2, 256, 256, 1e4, False, True, True, "16384"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _blocks(rng, rows):
    """rows packed rows: one causal block, or a prefix with ragged branches."""
    if rows < 4 or rng.random() < 0.3:
        return str(rows)
    cuts = sorted(rng.randint(0, rows) for _ in range(rng.randint(1, 6)))
    edges = [0] + cuts + [rows]
    return ",".join(str(b - a) for a, b in zip(edges, edges[1:]))


def draw(rng):
    head_dim = rng.choice([64, 128, 256, 512])
    n_kv = rng.choice([1, 2, 4])
    group = rng.choice([1, 2, 4, 8, 16])
    while n_kv * group * head_dim > 8192:
        group //= 2
    if rng.random() < 0.6:
        rows = _log(rng, 1, 4096)
        window = rng.choice([0, 0, _log(rng, 1, 2048)])
        return {k: v for k, v in _read("", n_kv * group, n_kv, head_dim, window, _blocks(rng, rows)).items()
                if k != "name"}
    rows = _log(rng, 1, 16384)
    while rows * n_kv * group * head_dim > 16384 * 2048:
        rows //= 2
    rope = rng.choice([0, head_dim // 4, head_dim // 2, head_dim])
    c = _prep("", n_kv * group, n_kv, head_dim, rope, rng.choice([1e4, 1e6]), rng.random() < 0.3, rng.random() < 0.7,
              rng.random() < 0.5, _blocks(rng, rows))
    return {k: v for k, v in c.items() if k != "name"}


def _sizes(case):
    return [int(b) for b in case["blocks"].split(",")]


def _visible_pairs(sizes, window):
    """(row, key) pairs of the layout: every row sees min(position + 1, window) keys."""
    total = 0
    for b, n in enumerate(sizes):
        first = 0 if b == 0 else sizes[0]
        if window <= 0 or first + n <= window:
            total += n * first + n * (n + 1) // 2
        else:
            grow = max(0, min(n, window - first))
            total += grow * first + grow * (grow + 1) // 2 + (n - grow) * window
    return total


def work(case):
    n, n_q, n_kv, d = sum(_sizes(case)), case["n_q"], case["n_kv"], case["head_dim"]
    if case["op"] == "read_backward":
        # q, dO, dq 2 bytes, out 4, lse 4 a row; k, v, dk, dv 2; five products over the visible pairs
        return {"bytes": n * n_q * (10 * d + 4) + n * n_kv * d * 8,
                "flops": 10.0 * d * n_q * _visible_pairs(_sizes(case), case["window"])}
    by = n * n_q * d * 6 + d * 6
    rows = n * n_q
    if case["donor"]:
        kinds = 1 if case["k_eq_v"] else 2
        by += n * n_kv * d * (kinds * 4 + 2 * (4 if case["kv_f32"] else 2)) + d * 6
        rows += 2 * n * n_kv
    return {"bytes": by, "flops": 12.0 * d * rows}


def _layout(sizes, device):
    """Block and position of every packed row, and the offsets."""
    n, t = sum(sizes), torch.tensor(sizes, device=device)
    block = torch.repeat_interleave(torch.arange(len(sizes), device=device), t)
    start = torch.cumsum(t, 0) - t
    pos = torch.arange(n, device=device) - start[block] + torch.where(block > 0, sizes[0], 0)
    offs = torch.cat([start, torch.tensor([n], device=device)]).to(torch.int32)
    return block, pos, offs


def _visible(block, pos, window):
    see = ((block[None, :] == 0) | (block[None, :] == block[:, None])) & (pos[None, :] <= pos[:, None])
    if window > 0:
        see &= pos[None, :] > pos[:, None] - window
    return see


def _heads_first(x, n_kv):
    """[rows, heads, D] -> [n_kv, group * rows, D] in 32 bits."""
    n, h, d = x.shape
    return x.float().reshape(n, n_kv, h // n_kv, d).permute(1, 2, 0, 3).reshape(n_kv, -1, d)


def _rows_first(x, n):
    """[n_kv, group * rows, D] -> [rows, heads, D]."""
    n_kv, gn, d = x.shape
    return x.reshape(n_kv, gn // n, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)


def _scores(state):
    """Masked scores [n_kv, group, rows, rows]."""
    n, n_kv = state["q"].shape[0], state["k"].shape[1]
    s = _heads_first(state["q"], n_kv) @ _heads_first(state["k"], n_kv).transpose(1, 2)
    see = _visible(state["block"], state["pos"], state["window"])
    return s.view(n_kv, -1, n, n).masked_fill_(~see, -math.inf)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    sizes = _sizes(case)
    n, n_q, n_kv, d = sum(sizes), case["n_q"], case["n_kv"], case["head_dim"]
    block, pos, offs = _layout(sizes, dev)
    state = {"case": dict(case), "block": block, "pos": pos, "offs": offs, "n_blocks": len(sizes),
             "max_rows": max(1, max(sizes))}
    if case["op"] == "read_backward":
        # normalised rows: heads from broad (scale 0.1) to sharp (scale 1: scores of deviation sqrt(D))
        scale = torch.linspace(0.1, 1.0, n_q, device=dev)[None, :, None]
        state["q"] = (rnd(n, n_q, d) * scale).bfloat16()
        state["k"], state["v"] = rnd(n, n_kv, d).bfloat16(), rnd(n, n_kv, d).bfloat16()
        state["d_out"] = (rnd(n, n_q, d) * 0.01).bfloat16()
        state["window"] = case["window"]
        # what the forward left: its output and each row's log-sum-exp
        s = _scores(state)
        lse = torch.logsumexp(s, -1)
        p = s.sub_(lse[..., None]).exp_()
        o = p.view(n_kv, -1, n) @ _heads_first(state["v"], n_kv)
        state["out"] = _rows_first(o, n).contiguous()
        state["lse"] = lse.permute(2, 0, 1).reshape(n, n_q).contiguous()
        return state
    state["q"], state["dq"] = rnd(n, n_q, d).bfloat16(), (rnd(n, n_q, d) * 0.01).bfloat16()
    state["q_w"], state["k_w"] = (1 + 0.1 * rnd(d)).bfloat16(), (1 + 0.1 * rnd(d)).bfloat16()
    if case["donor"]:
        kind = torch.float32 if case["kv_f32"] else torch.bfloat16
        state["k"] = rnd(n, n_kv, d).bfloat16()
        state["v"] = None if case["k_eq_v"] else rnd(n, n_kv, d).bfloat16()
        state["dk"], state["dv"] = (rnd(n, n_kv, d) * 0.01).to(kind), (rnd(n, n_kv, d) * 0.01).to(kind)
    return state


def _read_plain(state):
    n, n_kv = state["q"].shape[0], state["k"].shape[1]
    q, k, v, do = (_heads_first(state[x], n_kv) for x in ("q", "k", "v", "d_out"))
    s = _scores(state).view(n_kv, -1, n)
    p = (s - s.amax(-1, keepdim=True)).exp_()
    p /= p.sum(-1, keepdim=True)
    dp = do @ v.transpose(1, 2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    return {"dq": _rows_first(ds @ k, n).bfloat16(),
            "dk": (ds.transpose(1, 2) @ q).transpose(0, 1).bfloat16().contiguous(),
            "dv": (p.transpose(1, 2) @ do).transpose(0, 1).bfloat16().contiguous()}


def _norm_backward(x, dy, w):
    """Gradients of y = x r w (r = 1 / sqrt(mean(x^2) + eps), in 32 bits) by the input and by the weight."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dw = (dy * (x * r)).double().sum((0, 1)).float()
    wdy = dy if w is None else dy * w.float()
    return r * wdy - x * (r * r * r) * (wdy * x).mean(-1, keepdim=True), dw


def _unrotate(dz, pos, rope_dims, theta):
    """The transposed rotation of the first rope_dims dims (pairs j, j + rope_dims / 2)."""
    dz = dz.float()
    if rope_dims == 0:
        return dz
    h, d = rope_dims // 2, dz.shape[-1]
    f = theta ** (-2.0 * torch.arange(h, dtype=torch.float64, device=dz.device) / d)
    a = pos.double()[:, None, None] * f
    c, s = a.cos().float(), a.sin().float()
    lo, hi = dz[..., :h], dz[..., h:rope_dims]
    return torch.cat([lo * c + hi * s, hi * c - lo * s, dz[..., rope_dims:]], -1)


def _prep_plain(state):
    case = state["case"]
    dq, dq_w = _norm_backward(state["q"], _unrotate(state["dq"], state["pos"], case["rope_dims"], case["theta"]),
                              state["q_w"])
    got = {"dq": dq.bfloat16(), "dq_w": dq_w}
    if case["donor"]:
        dk, got["dk_w"] = _norm_backward(state["k"], _unrotate(state["dk"], state["pos"], case["rope_dims"],
                                                               case["theta"]), state["k_w"])
        dv, _ = _norm_backward(state["k"] if case["k_eq_v"] else state["v"], state["dv"].float(), None)
        if case["k_eq_v"]:
            got["dk"] = (dk + dv).bfloat16()
        else:
            got["dk"], got["dv"] = dk.bfloat16(), dv.bfloat16()
    return got


def _layer(kvq, case):
    return kvq.layer(case["n_q"], case["n_kv"], case["head_dim"], case.get("window", 0), case.get("rope_dims", 0),
                     case.get("theta", 1e4), EPS, case.get("k_eq_v", False))


def _read_own(state):
    import quantized_kv_attention_quant_gb300 as kvq
    n = state["q"].shape[0]
    if "lay" not in state:
        state["lay"] = _layer(kvq, state["case"])
        state["ws_bytes"] = kvq.attn_train_backward_workspace_bytes(state["lay"], state["n_blocks"], n,
                                                                    state["max_rows"])
        state["ws"] = torch.empty(state["ws_bytes"], dtype=torch.uint8, device="cuda")
        state["grads"] = {"dq": torch.empty_like(state["q"]), "dk": torch.empty_like(state["k"]),
                          "dv": torch.empty_like(state["v"])}
    g = state["grads"]
    kvq.attn_train_backward(state["lay"], state["n_blocks"], state["offs"], n, state["max_rows"], state["q"],
                            state["k"], state["v"], state["out"], 1, state["lse"], state["d_out"], g["dq"], g["dk"],
                            g["dv"], 0, 0, state["ws"], state["ws_bytes"])
    return g


def _prep_own(state):
    import quantized_kv_attention_quant_gb300 as kvq
    case, n, d = state["case"], state["q"].shape[0], state["q"].shape[2]
    donor, kv_f32 = case["donor"], int(case["kv_f32"])
    if "lay" not in state:
        state["lay"] = _layer(kvq, case)
        state["ws_bytes"] = kvq.kvq_train_prep_backward_workspace_bytes(state["lay"], n)
        state["ws"] = torch.empty(state["ws_bytes"], dtype=torch.uint8, device="cuda")
        g = {"dq": torch.empty_like(state["q"]), "dq_w": torch.empty(d, device="cuda")}
        if donor:
            g["dk"], g["dk_w"] = torch.empty_like(state["k"]), torch.empty(d, device="cuda")
            if not case["k_eq_v"]:
                g["dv"] = torch.empty_like(state["v"])
        state["grads"] = g
    g = state["grads"]
    kvq.kvq_train_prep_backward(state["lay"], state["n_blocks"], state["offs"], n, state["q"], state["q_w"],
                                state["dq"], g["dq"], g["dq_w"], state.get("k"), state.get("v"),
                                state["k_w"] if donor else None, state.get("dk"), state.get("dv"), kv_f32,
                                g.get("dk"), g.get("dv"), g.get("dk_w"), state["ws"], state["ws_bytes"])
    return g


def run(state):
    if state["case"]["op"] == "read_backward":
        return _read_own(state) if own else _read_plain(state)
    return _prep_own(state) if own else _prep_plain(state)


def exact(case, seed):
    """The definition in 64 bits, block by block and kv head by kv head."""
    state = prepare(case, seed)
    f = lambda x: state[x].double()  # noqa: E731
    sizes, n_kv = _sizes(case), case["n_kv"]
    group, p0 = case["n_q"] // n_kv, sizes[0]
    if case["op"] == "read_backward":
        q, k, v, do = f("q"), f("k"), f("v"), f("d_out")
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        at = 0
        for b, rows in enumerate(sizes):
            if rows:
                # the block's rows and the keys they may see: the prefix, then the block itself
                mine = torch.arange(at, at + rows, device="cuda")
                keys = mine if b == 0 else torch.cat([torch.arange(p0, device="cuda"), mine])
                i = torch.arange(rows, device="cuda")[:, None] + (0 if b == 0 else p0)
                j = torch.arange(len(keys), device="cuda")[None, :]
                hide = (j > i) if case["window"] <= 0 else (j > i) | (j <= i - case["window"])
                for h in range(case["n_q"]):
                    kv = h // group
                    s = torch.einsum("id,jd->ij", q[mine, h], k[keys, kv])
                    p = torch.softmax(s.masked_fill(hide, -math.inf), 1)
                    dp = torch.einsum("id,jd->ij", do[mine, h], v[keys, kv])
                    ds = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None])
                    dq[mine, h] = torch.einsum("ij,jd->id", ds, k[keys, kv])
                    dk[keys, kv] += torch.einsum("ij,id->jd", ds, q[mine, h])
                    dv[keys, kv] += torch.einsum("ij,id->jd", p, do[mine, h])
            at += rows
        return {"dq": dq, "dk": dk, "dv": dv}

    place = torch.cat([torch.arange(r, device="cuda") + (0 if b == 0 else p0) for b, r in enumerate(sizes)]).double()

    def through(x, dz, w, rotated):
        """d/dx and d/dw of sum(dz . R(norm(x) w)), by the Jacobian of each step."""
        d, half = x.shape[-1], case["rope_dims"] // 2
        dy = dz.clone()
        if rotated and half:
            rate = torch.tensor([case["theta"] ** (-2.0 * t / d) for t in range(half)], dtype=torch.float64,
                                device="cuda")
            z = torch.complex(dz[..., :half], dz[..., half:2 * half]) * torch.exp(-1j * place[:, None, None] * rate)
            dy[..., :half], dy[..., half:2 * half] = z.real, z.imag
        size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS)
        unit = x / size
        along = (dy * w * unit).sum(-1, keepdim=True) / d
        return (dy * w - unit * along) / size, (dy * unit).sum(0).sum(0)

    one = torch.ones(case["head_dim"], dtype=torch.float64, device="cuda")
    dq, dq_w = through(f("q"), f("dq"), f("q_w"), True)
    got = {"dq": dq, "dq_w": dq_w}
    if case["donor"]:
        dk, got["dk_w"] = through(f("k"), f("dk"), f("k_w"), True)
        dv, _ = through(f("k" if case["k_eq_v"] else "v"), f("dv"), one, False)
        if case["k_eq_v"]:
            got["dk"] = dk + dv
        else:
            got["dk"], got["dv"] = dk, dv
    return got
