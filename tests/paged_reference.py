"""Plain 64-bit forms of the paged cache's operators, for the tests: attention
over pages by direct summation, and the page bookkeeping as loops over lists."""
import math

import torch


def attention(q, k_pages, v_pages, table, lens, scale, window=-1):
    """O and LSE in fp64, and error bounds for a kernel with bf16 products, fp32
    sums and weights rounded to bf16 (see `bounds`).

    q [B, H, T, D]; k_pages [P, Hkv, page, D]; v_pages [P, Hkv, page, Dv]."""
    B, H, T, D = q.shape
    P, Hkv, page, Dv = v_pages.shape
    dev = q.device
    o = torch.zeros((B, H, T, Dv), dtype=torch.float64, device=dev)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=dev)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    cap = table.shape[1] * page
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        if n == 0:
            continue
        ids = table[b, : -(-n // page)].long()
        good = (ids >= 0) & (ids < P)
        slots = good.repeat_interleave(page)[:n]
        ids = torch.where(good, ids, 0)
        k = torch.where(slots[None, :, None], k_pages[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :n], 0).double()
        v = torch.where(slots[None, :, None], v_pages[ids].transpose(0, 1).reshape(Hkv, -1, Dv)[:, :n], 0).double()
        at = torch.arange(n, device=dev)
        for u in range(T):
            last = n - T + u
            seen = slots & (at <= last)
            if window >= 0:
                seen &= at >= last - window
            if not bool(seen.any()):
                continue
            kk, vv = k[:, seen], v[:, seen]
            qq = q[b, :, u].double().view(Hkv, H // Hkv, D)
            s = torch.matmul(qq, kk.transpose(1, 2)) * scale
            w = torch.softmax(s, -1)
            lse[b, :, u] = torch.logsumexp(s, -1).reshape(H)
            o[b, :, u] = torch.matmul(w, vv).reshape(H, Dv)
            # the sums of the products' sizes, for the bounds
            size = (torch.matmul(qq.abs(), kk.abs().transpose(1, 2)) * scale).amax(-1).reshape(H)
            wide = torch.matmul(w, vv.abs()).reshape(H, Dv)
            eo[b, :, u], el[b, :, u] = bounds(o[b, :, u], lse[b, :, u], size, wide, D, int(seen.sum()))
    return o, lse, eo, el


def bounds(o, lse, size, wide, D, n):
    """How far a kernel may be from o and lse.

    A score of D products summed in fp32 (2^-23 an addition where the hardware
    truncates) is off by es = (D + 4) 2^-23 size, size the sum of the products'
    absolute values; scaling, the exponent's argument and the exponential add a
    few 2^-23 of their own, of the score's size. A weight is then off by the
    factor 1 + es, and the normaliser's sum of n terms, at most n / 64 + 64
    deep, by (n / 64 + 64) 2^-24. Weights are rounded to bf16 (half a step,
    2^-8) before the value products, whose fp32 sums add a like (n + 64) 2^-23
    at worst of `wide` = sum w |v|; O is rounded to bf16 once. 1.02 covers the
    second-order terms."""
    es = (D + 16) * 2.0 ** -23 * size + 2.0 ** -21
    ed = (n / 64 + 64) * 2.0 ** -24
    rel = 2.0 ** -8 + 2 * es + ed + min(n + 64, 4096) * 2.0 ** -23
    eo = 1.02 * (rel[:, None] * wide + 2.0 ** -8 * o.abs()) + 1e-30
    el = 1.02 * (es + ed + 2.0 ** -22 * (lse.abs() + 1))
    return eo, el


def check(o, lse, ref):
    """The kernel's o and lse within the bounds of `attention`'s answer."""
    ro, rl, eo, el = ref
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse.double()), empty), "rows without a position"
    assert torch.isfinite(o.float()).all()
    assert (o[empty] == 0).all()
    dl = (lse.double() - rl).abs()[~empty]
    assert (dl <= el[~empty]).all(), f"LSE off by {(dl / el[~empty]).max().item():.3f} of its bound"
    do = (o.double() - ro).abs()
    assert (do <= eo).all(), f"O off by {(do / eo.clamp(min=1e-300)).max().item():.3f} of its bound"


class Pages:
    """The bookkeeping as plain lists."""

    def __init__(self, table, lens, refs, page):
        self.table = [list(map(int, r)) for r in table]
        self.lens, self.refs, self.page = [int(x) for x in lens], [int(x) for x in refs], page

    def free_pages(self):
        return [p for p, n in enumerate(self.refs) if n <= 0]

    def is_page(self, e):
        return 0 <= e < len(self.refs)

    def reserve(self, rows, want):
        free, granted, asked, seen = self.free_pages(), [], 0, set()
        for r, w in zip(rows, want):
            bad = not 0 <= r < len(self.table) or r in seen or w > len(self.table[0]) * self.page
            if 0 <= r < len(self.table):
                seen.add(r)
            if bad:
                granted.append(0)
                continue
            empty = [j for j in range(-(-max(w, 0) // self.page)) if not self.is_page(self.table[r][j])]
            first, asked = asked, asked + len(empty)
            granted.append(int(not empty or asked <= len(free)))
            if granted[-1]:
                for j, p in zip(empty, free[first:asked]):
                    self.table[r][j] = p
                    self.refs[p] = 1
        return granted

    def fork(self, parents, children):
        """(fresh, granted, copies): copies are (from page, to page, rows)."""
        free, fresh, granted, copies, asked, seen = self.free_pages(), [], [], [], 0, set()
        before_len, before = list(self.lens), [list(r) for r in self.table]
        R, width = len(self.table), len(self.table[0])
        for f, c in zip(parents, children):
            ok = 0 <= f < R and 0 <= c < R and c not in seen and before_len[c] == 0 and not self.is_page(before[c][0])
            if 0 <= c < R:
                seen.add(c)
            ok = ok and before_len[f] <= width * self.page
            page = -1
            if ok:
                n = max(before_len[f], 0)
                full, part = divmod(n, self.page)
                last = before[f][full] if part else -1
                if part and self.is_page(last):
                    asked += 1
                    if asked <= len(free):
                        page = free[asked - 1]
                    else:
                        ok = False
            fresh.append(page)
            granted.append(int(ok))
            if ok:
                self.table[c] = before[f][:full] + [-1] * (width - full)
                if full < width:
                    self.table[c][full] = page
                self.lens[c] = n
                for e in before[f][:full]:
                    if self.is_page(e):
                        self.refs[e] += 1
                if page >= 0:
                    self.refs[page] = 1
                    copies.append((last, page, part))
        return fresh, granted, copies

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table):
                for e in self.table[r]:
                    if self.is_page(e):
                        self.refs[e] -= 1
                self.table[r] = [-1] * len(self.table[r])
                self.lens[r] = 0

    def compact(self):
        """(live, moves): moves are (from page, to page)."""
        live = sum(n > 0 for n in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        name = dict(zip(movers, holes))
        self.table = [[name.get(e, e) for e in r] for r in self.table]
        for a, b in name.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.refs = [max(n, 0) for n in self.refs]
        return live, list(name.items())
