"""How the packed attention's plan cuts items into parts (csrc/packed_plan.cu), restated on the CPU:
for tests of its bound on the parts' number, and for finding calls that reach a branch of it."""
import numpy as np

TILE, LEAST_PART, LEAST_CUT = 128, 4, 8
MAX_PARTS = {"fwd": 320, "bwd": 512}
MANY_ITEMS = 1024
SMS = 152


def slots_of(which, T, n, Hq, Hk):
    """Slots of a key head in the call's workspace."""
    tq = TILE // (Hq // Hk)
    if which == "fwd":
        items = T // (2 * tq) + n
        most = 0 if T <= TILE * LEAST_CUT or items * Hk >= MANY_ITEMS else \
            items * (T // TILE // LEAST_PART + 1)
    else:
        most = 0 if (T - 1) // tq + 1 <= LEAST_CUT else \
            (T // TILE + n) * (T // tq // LEAST_PART + 1)
    slots = min(most, -(-MAX_PARTS[which] // Hk))
    return 0 if slots < 3 else slots


def cut(which, lens, T, Hq, Hk, causal, sms=SMS):
    """The slots, the items of a key head, the tiles that each streams, the length of a part, and
    whether that is the bound's and not the share's."""
    tq = TILE // (Hq // Hk)
    tokens = TILE if which == "bwd" else 2 * tq
    slots = slots_of(which, T, len(lens), Hq, Hk)
    streamed, estimate = [], 0.0
    for n in map(int, lens):
        tiles = -(-n // tokens)
        if tiles == 0:
            continue
        z = np.arange(tiles)
        if which == "bwd":
            streamed.append((n - 1) // tq - (z * TILE // tq if causal else 0 * z) + 1)
            some = tiles * ((n - 1) // tq + 1)
            if causal:
                some -= max(0.0, tiles * (tiles - 1) * (0.5 * TILE) / tq - tiles)
        else:
            seen = np.minimum((z + 1) * tokens, n) if causal else n + 0 * z
            streamed.append((seen - 1) // TILE + 1)
            some = tiles * ((n - 1) // TILE + 1)
            if causal:
                some = min(some, tiles * (tiles + 1) * (0.5 / TILE) * tokens + tiles)
        estimate += some
    streamed = np.concatenate(streamed) if streamed else np.zeros(0, dtype=int)
    items = len(streamed)
    if slots == 0 or items == 0:
        return slots, items, streamed, None, False
    total = 1.001 * estimate
    mean = total * Hk / sms
    down = 0.45 if which == "bwd" and items * Hk <= sms else 0.6
    share = down * mean + min((1.3 - down) * mean, 20.0)
    least = total / (slots - items) if 2 * items < slots else 2 * total / slots
    return (slots, items, streamed, max(LEAST_PART, int(max(share, least) + 1)), least > share)


def parts(streamed, chunk):
    """Parts of the items that are cut."""
    n = streamed[(streamed > LEAST_CUT) & (streamed > chunk)]
    return int(((n - 1) // chunk + 1).sum())
