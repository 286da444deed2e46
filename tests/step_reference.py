"""A step's bookkeeping in Python integers, one block and one row at a time: what
plan_step, release_blocks and commit_tokens define."""


class Step:
    """State (tables, held, the stack of free blocks) and the arrays of one step."""

    def __init__(self, tables, held, stack, block):
        self.tables = [list(map(int, t)) for t in tables]
        self.held = [int(h) for h in held]
        self.stack = [int(b) for b in stack]
        self.block = block

    def plan(self, ctx, new, max_tokens, parents=None, words=0):
        B, S = self.block, len(ctx)
        width = len(self.tables[0]) if S else 0
        ok = [n >= 0 and c >= 0 and (words == 0 or n <= 64 * words) and c + n <= width * B and
              0 <= h <= width for c, n, h in zip(ctx, new, self.held)]
        first = [0]
        for n in new:
            first.append(first[-1] + max(n, 0))
        need = sum(max(0, -(-(c + n) // B) - h) for c, n, h, o in zip(ctx, new, self.held, ok) if o)
        fits = first[-1] <= max_tokens and need <= len(self.stack)
        seq = [0] * S
        slots, positions = [-1] * max_tokens, [0] * max_tokens
        masks = [0] * max_tokens
        for r in range(S):
            if not (ok[r] and fits):
                continue
            seq[r] = ctx[r] + new[r]
            while self.held[r] * B < seq[r]:
                self.tables[r][self.held[r]] = self.stack.pop()
                self.held[r] += 1
            for i in range(new[r]):
                t = first[r] + i
                slots[t] = self.tables[r][(ctx[r] + i) // B] * B + (ctx[r] + i) % B
                node, depth, bits = i, 0, 1 << i
                while True:
                    up = node - 1 if parents is None else parents[first[r] + node]
                    if up < 0:
                        break
                    node, depth, bits = up, depth + 1, bits | 1 << up
                positions[t] = ctx[r] + depth
                masks[t] = bits
        return dict(qsl=first, seq=seq, slots=slots, positions=positions, masks=masks)

    def release(self, keep):
        """The blocks behind keep, those of the last request and position first."""
        for r in reversed(range(len(keep))):
            while self.held[r] > -(-keep[r] // self.block):
                self.held[r] -= 1
                self.stack.append(self.tables[r][self.held[r]])


def words_of(masks, words):
    """Rows of signed 64-bit words of arbitrary integers."""
    out = []
    for m in masks:
        row = [(m >> 64 * w) & ((1 << 64) - 1) for w in range(words)]
        out.append([x - (1 << 64) if x >> 63 else x for x in row])
    return out
