"""A paged 8-bit cache in plain numpy: quantized rows and scales as the header
defines them (IEEE fp32 where it says so), attention over them in float64, and
the pool's bookkeeping one sequence and one page after another."""
import numpy as np

import oracle as O

F32 = np.float32
TOP = {"i8": 127.0, "e4m3": 448.0}


def _e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


E4M3 = _e4m3_table()


def code_values(raw, kind):
    """float64 values of code bytes (uint8)."""
    return raw.view(np.int8).astype(np.float64) if kind == "i8" else E4M3[raw]


def encode(q, kind):
    """Code bytes of float32 quotients."""
    q = q.astype(np.float64)
    if kind == "i8":
        return np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    _, e = np.frexp(q)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    v = np.clip(np.rint(q / step) * step, -448, 448)
    mag = np.abs(v)
    order = np.argsort(E4M3[:127], kind="stable")
    at = np.searchsorted(E4M3[:127][order], mag)
    b = order[at].astype(np.uint8)
    return (b | (np.signbit(v).astype(np.uint8) << 7)).astype(np.uint8)


class Pages:
    """One layer's pages, filled with bytes that no read may use."""

    def __init__(self, n_pages, n_kv, P, D, kind, seed=0, fill=None):
        g = np.random.default_rng(seed)
        self.n_pages, self.n_kv, self.P, self.D, self.kind = n_pages, n_kv, P, D, kind
        shape = (n_pages, n_kv, P, D)
        blank = (lambda: np.full(shape, fill, np.uint8)) if fill is not None else \
            (lambda: g.integers(0, 256, shape, dtype=np.uint8))
        self.codes = {"k": blank(), "v": blank()}
        self.scales = {c: np.full((n_pages, n_kv), np.nan, F32) for c in "kv"}

    def append(self, table, start, k_hat, v_hat):
        """Rows [rows, n_kv, D] (float64 values of bf16) at positions start .. of the sequence with this table."""
        for c, x in (("k", k_hat), ("v", v_hat)):
            rows, p = x.shape[0], start
            while p < start + rows:
                i, end = p // self.P, min(start + rows, (p // self.P + 1) * self.P)
                page, slot, new = table[i], p % self.P, x[p - start:end - start].astype(F32)
                for h in range(self.n_kv):
                    top = F32(np.abs(new[:, h]).max())
                    s = F32(top / F32(TOP[self.kind]))
                    s = F32(0) if s < F32(2.0 ** -40) else s
                    if slot:
                        was = self.scales[c][page, h]
                        if s > was:
                            old = code_values(self.codes[c][page, h, :slot], self.kind).astype(F32)
                            self.codes[c][page, h, :slot] = encode((old * was).astype(F32) / s, self.kind)
                        s = max(s, was)
                    q = new[:, h] / s if s > 0 else np.zeros_like(new[:, h])
                    self.codes[c][page, h, slot:slot + end - p] = encode(q, self.kind)
                    self.scales[c][page, h] = s
                p = end

    def values(self, c, table, h, positions):
        """float64 values code * scale of a head's rows."""
        pos = np.asarray(positions)
        page = np.asarray(table)[pos // self.P]
        return code_values(self.codes[c][page, h, pos % self.P], self.kind) * \
            self.scales[c][page, h].astype(np.float64)[:, None]


def attend(pages, table, q_hat, p, window):
    """q_hat [n_q, D] at position p -> the output, and for each output the weighted sum of |v| and the row's
    largest sum of |q k| over its keys (what the bound of its rounding scales with)."""
    n_q, D = q_hat.shape
    G = n_q // pages.n_kv
    keys = np.arange(max(0, p - window + 1) if window > 0 else 0, p + 1)
    out, mag, big = np.zeros((n_q, D)), np.zeros((n_q, D)), np.zeros((n_q, 1))
    for h in range(pages.n_kv):
        k, v = pages.values("k", table, h, keys), pages.values("v", table, h, keys)
        q = q_hat[h * G:(h + 1) * G]
        s = q @ k.T
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[h * G:(h + 1) * G] = w @ v
        mag[h * G:(h + 1) * G] = w @ np.abs(v)
        big[h * G:(h + 1) * G, 0] = (np.abs(q) @ np.abs(k).T).max(1)
    return out, mag, big


def bound(out, mag, big, n_keys, D, out_bf16):
    """How far an output may be off.  Each probability is rounded to f16 (2^-11 of it; those below f16's normal range,
    2^-14 against at least 2^7 of the largest term, by 2^-25 / 2^7 of the largest weight each).  A score is a sum of
    exact products, fp32 with at most 2^-23 of the running magnitude lost at each of its D/16 steps and a few more in
    scaling and exponent: an error d multiplies a probability by e^d, in the sums above and below the line (2 d).  The
    sums over the keys lose 2^-23 of the running magnitude per 16 keys.  The result is rounded once."""
    d = (D / 16 + 16) * 2.0 ** -23 * big + 2.0 ** -20
    rel = 2.0 ** -11 + 2 * d + (n_keys / 16 + 64) * 2.0 ** -23
    tiny = n_keys * 2.0 ** -32 * mag.max(1, keepdims=True) * 16
    return 1.001 * (rel * mag + tiny + (2.0 ** -8 if out_bf16 else 2.0 ** -24) * np.abs(out)) + 1e-30


def prep(q_raw, w, pos, layer):
    """Prepped rows of bf16 bit patterns [rows, heads, D] (w None: the un-scaled norm without rotation)."""
    eps = float(np.float32(layer.rms_eps))
    x = O.bf16_to_f64(q_raw)
    if w is None:
        return O.prep_v(x, eps)
    return O.prep_q(x, O.bf16_to_f64(w), np.asarray(pos), layer.rope_theta, layer.rope_dims, eps)


class Pool:
    """The pool's bookkeeping as the header defines it."""

    def __init__(self, n_seqs, max_pages, n_pages, P):
        self.P, self.max_pages = P, max_pages
        self.tables = [[-1] * max_pages for _ in range(n_seqs)]
        self.lens, self.refs = [0] * n_seqs, [0] * n_pages

    def held(self, s):
        return -(-self.lens[s] // self.P)

    def free(self, seqs, keep=None):
        done = set()
        for i, s in enumerate(seqs):
            if s in done or not 0 <= s < len(self.lens):
                continue
            done.add(s)
            left = min(self.lens[s], max(0, keep[i]) if keep is not None else 0)
            for k in range(-(-left // self.P), self.held(s)):
                self.refs[self.tables[s][k]] -= 1
                self.tables[s][k] = -1
            self.lens[s] = left

    def fork(self, parents, children):
        granted, n = [], len(self.lens)
        before = list(self.lens)
        for i, (a, b) in enumerate(zip(parents, children)):
            ok = 0 <= a < n and 0 <= b < n and a not in children and b not in children[:i] and before[b] == 0
            granted.append(int(ok))
            if ok:
                self.lens[b] = self.lens[a]
                for k in range(self.held(a)):
                    self.tables[b][k] = self.tables[a][k]
                    self.refs[self.tables[a][k]] += 1
        return granted

    def reserve(self, n_new):
        """Granted, start positions and the (source, destination) copies."""
        free, before = [i for i, r in enumerate(self.refs) if r == 0], list(self.refs)
        granted, start, copies, asked = [], list(self.lens), [], 0
        for s, n in enumerate(n_new):
            to = self.lens[s] + max(0, n)
            if to > self.max_pages * self.P or to > 1 << 24:
                granted.append(0)
                continue
            have, want = self.held(s), -(-to // self.P)
            shared = n > 0 and self.lens[s] % self.P and before[self.tables[s][have - 1]] > 1
            need = want - have + bool(shared)
            mine = free[asked:asked + need]
            asked += need
            granted.append(int(len(mine) == need))
            if len(mine) < need:
                continue
            if shared:
                copies.append((self.tables[s][have - 1], mine[0]))
                self.refs[self.tables[s][have - 1]] -= 1
                self.tables[s][have - 1] = mine.pop(0)
                self.refs[self.tables[s][have - 1]] = 1
            for k, page in zip(range(have, want), mine):
                self.tables[s][k] = page
                self.refs[page] = 1
            self.lens[s] = to
        return granted, start, copies

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [i for i in range(live) if self.refs[i] == 0]
        late = [i for i in range(live, len(self.refs)) if self.refs[i] > 0]
        to = [i if r > 0 else -1 for i, r in enumerate(self.refs)]
        for a, b in zip(late, holes):
            to[a], self.refs[b], self.refs[a] = b, self.refs[a], 0
        for s in range(len(self.lens)):
            for k in range(self.held(s)):
                self.tables[s][k] = to[self.tables[s][k]]
        return live, to, list(zip(late, holes))
