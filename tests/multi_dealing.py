"""How the attention of several new tokens deals its work out where the host
chose equal shares of all tiles, restated in Python: which segments each CTA
gets, which states it writes and what the join reads.  Tests use it to name
shapes by what they reach and to check the indexes for them."""

TILE, ITEM_ROWS, SLOT_ROWS = 128, 256, 128


class Dealing:
    """n: new tokens, T: lengths (one entry per sequence), as the kernel sees
    them after its clamps; G heads per group; tree: ancestor mask."""

    def __init__(self, n, T, hkv, G, tree, max_new=None, n_tokens=None, ctas=148):
        self.hkv, self.tree, self.ctas = hkv, tree, ctas
        self.tpi, self.tps = ITEM_ROWS // G, SLOT_ROWS // G
        self.n, self.T = list(n), list(T)
        max_new = max_new or max(n)
        self.kept = [min(x, max_new) for x in n]
        tokens = sum(n) if n_tokens is None else n_tokens
        self.item_bound = min(tokens // self.tpi + len(n), len(n) * -(-max_new // self.tpi))
        self.by_item = self.item_bound * hkv <= ctas
        self.line = []  # (sequence, item, head, tiles, unit, first unit on the line)
        at = 0
        self.items_before = []
        items_before = 0
        for b, kept in enumerate(self.kept):
            self.items_before.append(items_before)
            items = -(-kept // self.tpi)
            for i in range(items):
                tiles, unit = self.tiles(b, i), self.unit(b, i)
                for g in range(hkv):
                    self.line.append((b, i, g, tiles, unit, at))
                    at += (tiles + 1) * unit if tiles else 0
            items_before += items
        self.total, self.items = at, items_before * hkv
        self.shares = max(1, min(ctas, at >> 5))
        self.each, self.rest = divmod(at, self.shares)
        self._deal()

    def upto(self, b, last):
        rows = self.T[b] if self.tree else min(self.T[b], self.T[b] - self.n[b] + last + 1)
        return max(0, -(-rows // TILE))

    def tiles(self, b, i):
        return self.upto(b, min((i + 1) * self.tpi, self.kept[b]) - 1)

    def unit(self, b, i):
        return 7 if min(self.tpi, self.kept[b] - i * self.tpi) > self.tps else 5

    def begin(self, c):
        return self.total if c >= self.shares else self.each * c + min(c, self.rest)

    def holding(self, u):
        big = (self.each + 1) * self.rest
        return u // (self.each + 1) if u < big else self.rest + (u - big) // self.each

    def _deal(self):
        """segments: (cta, sequence, item, head, first tile, last, tiles of slot
        0, state written or -1); joins: entry -> (first CTA or -1, CTAs)."""
        self.segments, self.joins = [], {}

        def behind(x, unit):
            return 0 if x == 0 else max(1, -(-x // unit) - 1)

        for c in range(self.ctas):
            w, w1, joined = self.begin(c), self.begin(c + 1), False
            for b, i, g, tiles, unit, at in self.line:
                end = at + ((tiles + 1) * unit if tiles else 0)
                if not (at <= w < end) or w >= w1:
                    continue
                first, last = behind(w - at, unit), min(tiles, behind(w1 - at, unit))
                w = min(end, w1)
                if first >= last:
                    continue
                ntok = min(self.tpi, self.kept[b] - i * self.tpi)
                pair = ntok > self.tps
                nt = last - first
                t0 = max(0, min(last, self.upto(b, i * self.tpi + self.tps - 1)) - first) if pair else (nt + 1) // 2
                whole = first == 0 and last == tiles
                self.segments.append((c, b, i, g, first, last, t0, -1 if whole else 2 * c + (first == 0)))
                if last == tiles and (first > 0 or self.by_item):
                    src = self.holding(at) if first > 0 else -1
                    self._join((self.items_before[b] + i) * self.hkv + g if self.by_item else c, src, c - src + 1)
                    joined = True
            if self.by_item:
                if self.items <= c < self.item_bound * self.hkv:
                    self._join(c, -1, 0)
            elif not joined:
                self._join(c, -1, 0)
        if self.by_item:
            for b, i, g, tiles, _, _ in self.line:
                if tiles == 0:
                    self._join((self.items_before[b] + i) * self.hkv + g, -1, 0)

    def _join(self, entry, src, n):
        assert entry not in self.joins, f"entry {entry} written twice"
        self.joins[entry] = (src, n)

    def check(self):
        """Every tile in one segment, every state that a join reads written by
        that item, every entry in the list and the whole list written."""
        seen, state = {}, {}
        for c, b, i, g, first, last, _, part in self.segments:
            for t in range(first, last):
                assert (b, i, g, t) not in seen
                seen[b, i, g, t] = c
            if part >= 0:
                assert 0 <= part < 2 * self.ctas and part not in state
                state[part] = (b, i, g)
        assert len(seen) == sum(tiles for _, _, _, tiles, _, _ in self.line)
        used = {e for e in self.joins}
        assert used == set(range(self.item_bound * self.hkv if self.by_item else self.ctas)), "list not written whole"
        read = set()
        for src, n in self.joins.values():
            if src < 0:
                continue
            parts = [2 * (src + s) + (s == 0) for s in range(n)]
            assert all(p in state for p in parts) and len({state[p] for p in parts}) == 1, (src, n)
            read |= set(parts)
        assert read == set(state)
        return self

    def slot0_without_tiles(self):
        """Segments of two row blocks of which the first has no tile."""
        return sum(1 for _, b, i, _, _, _, t0, _ in self.segments
                   if t0 == 0 and min(self.tpi, self.kept[b] - i * self.tpi) > self.tps)
