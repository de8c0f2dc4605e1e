"""Which workgroup of paged_attn's launches writes what into the workspace:
its plan and its kernels' block numbers and places of partial results, redone
in plain whole numbers."""

from types import SimpleNamespace

UNIT = 128


def up(a, b):
    return -(-a // b)


def plan(T, B, Hq, Hkv, D, keys, prefix):
    G = Hq // Hkv
    rows, wide, p = T * G, 16 * (1 if D == 256 else 2), SimpleNamespace()

    def splits(blocks, waves, most):
        want, tiles = up(2048 // waves, blocks * Hkv), up(most, 256)
        return want if want < tiles else max(tiles, 1)

    blocks = up(rows, 16) * Hkv
    if rows > 48 * B:
        p.own_wide = blocks > 512 or up(keys, UNIT) * blocks > 6144
    else:
        p.own_wide = rows > 16 * B and blocks > 512 and keys <= 256
    p.pre_wide = prefix > 0 and (p.own_wide or up(prefix, UNIT) * blocks > 4096)
    p.own_waves, p.pre_waves = (8 if rows >= 1024 * B else 4), (8 if rows >= 1024 else 4)
    p.own_rows = wide * p.own_waves if p.own_wide else 16
    p.pre_rows = wide * p.pre_waves if p.pre_wide else 16
    p.own_blocks = rows // p.own_rows + B
    p.pre_blocks = up(rows, p.pre_rows) if prefix else 0
    p.own_splits = p.pre_splits = p.own_groups = p.pre_slots = 0
    p.complete = False
    if p.own_wide:
        p.own_splits = splits(p.own_blocks, p.own_waves, keys)
        p.complete = p.own_splits == 1 and prefix == 0
        p.own_slots = p.own_blocks * Hkv * p.own_splits
    else:
        most = max(1, up(keys, UNIT) * (rows // 16 + B) * Hkv +
                   (0 if p.pre_wide else up(prefix, UNIT) * p.pre_blocks * Hkv))
        p.own_groups = min(most, 768)
        p.own_slots = p.own_groups + (p.own_blocks + (0 if p.pre_wide else p.pre_blocks)) * Hkv
    if p.pre_wide:
        p.pre_splits = splits(p.pre_blocks, p.pre_waves, prefix)
        p.pre_slots = p.pre_blocks * Hkv * p.pre_splits
        p.own_slots = up(p.own_slots * p.own_rows, p.pre_rows) * p.pre_rows // p.own_rows
    p.partial_rows = p.own_slots * p.own_rows + p.pre_slots * p.pre_rows
    aligned = lambda v: (v + 255) & ~255
    p.off_ml = aligned((p.own_blocks + p.pre_blocks) * Hkv * 8)
    p.off_part = p.off_ml + aligned(p.partial_rows * 8)
    p.bytes = p.off_part + (0 if p.complete else p.partial_rows * D * 4)
    return p


class Writes:
    """What the launches of one call write: per block number (block and key
    head) the pair (first place, count or -1), and the places of partial results
    with their number of rows."""

    def __init__(self, p, T, Hq, Hkv, start, lens, window, prefix, D, groups=None):
        self.p, self.T, self.G, self.Hkv = p, T, Hq // Hkv, Hkv
        self.prefix, self.window, self.D = prefix, window, D
        self.seqs = []
        for b, n in enumerate(lens):
            q0 = min(max(start[b], 0), T)
            self.seqs.append((q0, min(max(start[b + 1], q0), T) - q0, n))
        self.meta, self.partials, self.direct = {}, [], set()
        if p.pre_wide:
            self.rows_launch(True)
        if p.own_wide:
            self.rows_launch(False)
        else:
            self.split_launch(min(groups or p.own_groups, p.own_groups))

    def base(self, b, rows):
        return self.seqs[b][0] * self.G // rows + b

    def put(self, id, pair):
        assert id not in self.meta
        self.meta[id] = pair

    def split_launch(self, groups):
        p, G, Hkv = self.p, self.G, self.Hkv
        segments = []                              # (units, id) of each block and key head
        for b, (q0, n, length) in enumerate(self.seqs):
            if n == 0 or length == 0:
                continue
            first = max(length - n - self.window + 1, 0) if self.window else 0
            units = up(length, UNIT) - first // UNIT
            assert units > 0
            for j in range(up(n * G, 16)):
                for h in range(Hkv):
                    segments.append((units, (self.base(b, 16) + j) * Hkv + h))
        if self.prefix and not p.pre_wide:
            for j in range(up(self.T * G, 16)):
                for h in range(Hkv):
                    segments.append((up(self.prefix, UNIT), (p.own_blocks + j) * Hkv + h))
        total = sum(u for u, _ in segments)
        per = up(total, groups)
        at = 0
        for units, id in segments:
            w0, w1 = at // per, (at + units - 1) // per
            direct = w0 == w1 and not self.prefix
            self.put(id, (w0 + id, -1 if direct else w1 - w0 + 1))
            if direct:
                self.direct.add(id)
            else:
                self.partials += [(id, w + id, 16) for w in range(w0, w1 + 1)]
            at += units

    def rows_launch(self, pre):
        p, G, Hkv = self.p, self.G, self.Hkv
        waves, rows = (p.pre_waves, p.pre_rows) if pre else (p.own_waves, p.own_rows)
        splits, blocks = (p.pre_splits, p.pre_blocks) if pre else (p.own_splits, p.own_blocks)
        tile = 2048 * waves // self.D
        for blk in range(blocks):
            first = 0
            if pre:
                end = up(self.prefix, tile)
            else:
                b = sum(self.base(i, rows) <= blk for i in range(len(self.seqs))) - 1
                if b < 0:
                    continue
                q0, n, length = self.seqs[b]
                j = blk - self.base(b, rows)
                if j < 0 or j * rows >= n * G:
                    continue
                live = min(rows, n * G - j * rows)
                pos0, pos1 = length - n + j * rows // G, length - n + (j * rows + live - 1) // G
                end = up(min(max(pos1 + 1, 0), length), tile)
                if self.window:
                    first = max(pos0 - self.window + 1, 0) // tile
            tiles = max(end - first, 0)
            per = up(tiles, splits)
            parts = up(tiles, per) if per else 0
            direct = not pre and parts <= 1 and not self.prefix
            for h in range(Hkv):
                id = ((p.own_blocks + blk) if pre else blk) * Hkv + h
                place = (blk * Hkv + h) * splits + (p.own_slots * p.own_rows // rows if pre else 0)
                self.put(id, (place, -1 if direct else parts))
                if direct:
                    self.direct.add(id)
                else:
                    self.partials += [(id, place + s, rows) for s in range(parts)]

    def joined(self, t, head):
        """(block number, row of the block, rows of a block) of the partial results a row's join reads."""
        p, G, h = self.p, self.G, head // self.G
        out = []
        for b, (q0, n, length) in enumerate(self.seqs):
            if q0 <= t < q0 + n and length > 0:
                local = (t - q0) * G + head % G
                out.append(((self.base(b, p.own_rows) + local // p.own_rows) * self.Hkv + h,
                            local % p.own_rows, p.own_rows))
        if self.prefix:
            row = t * G + head % G
            out.append(((p.own_blocks + row // p.pre_rows) * self.Hkv + h, row % p.pre_rows, p.pre_rows))
        return out
