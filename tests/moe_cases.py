"""Sizes that reach each kernel of the 8-bit products: (kind, tile rows, tile columns, split) of the plan for 256
compute units, rows by expert, rows before the first, rows after the last, N, K, MiB of workspace."""
MIB = 1 << 20


def shares(T, E, seed):
    """T rows by E experts, uneven, some of none."""
    w = [((seed + 7) * (e + 3) * (e + 11)) % 97 if (e + seed) % 5 else 0 for e in range(E)]
    w[E // 2] += 40
    n = [T * x // sum(w) for x in w]
    n[E // 2] += T - sum(n)
    return n


def _case(kind, T, E, N, K, mib, lead=0, tail=0):
    return kind, shares(T - lead - tail, E, T + N), lead, tail, N, K, mib


PRODUCTS = [
    _case(("ring", 16, 64, False), 13, 1, 72, 4096, 0, 2, 3),
    _case(("ring", 16, 64, False), 137, 13, 72, 2064, 0),
    _case(("ring", 16, 64, True), 37, 3, 1032, 8208, 4, 0, 1),
    _case(("ring", 16, 64, True), 137, 13, 520, 4112, 4),
    _case(("ring", 32, 64, False), 3, 1, 40, 80, 0),
    _case(("ring", 32, 64, False), 531, 40, 264, 528, 0, 3, 2),
    _case(("ring", 32, 64, True), 13, 1, 40, 2064, 4),
    _case(("ring", 32, 64, True), 1013, 7, 40, 8208, 4, 0, 5),
    _case(("ring", 64, 64, False), 2021, 13, 520, 272, 0, 1, 1),
    _case(("ring", 64, 64, False), 4111, 40, 136, 8208, 0),
    _case(("ring", 64, 64, True), 1013, 40, 72, 4112, 4),
    _case(("ring", 64, 64, True), 2021, 3, 136, 8208, 4, 2, 0),
    _case(("ring", 64, 128, False), 531, 13, 4104, 80, 0),
    _case(("ring", 64, 128, False), 2021, 7, 520, 8208, 0, 5, 0),
    _case(("ring", 64, 128, True), 531, 13, 264, 8208, 4, 0, 9),
    _case(("ring", 64, 128, True), 4111, 40, 72, 8208, 4),
    _case(("ring", 128, 64, False), 2021, 3, 1032, 144, 0),
    _case(("ring", 128, 64, False), 4111, 13, 264, 4096, 0, 7, 3),
    _case(("ring", 128, 64, True), 13, 1, 40, 4096, 4, 1, 0),
    _case(("ring", 128, 64, True), 2021, 70, 40, 4096, 4),
    _case(("ring", 128, 128, False), 1013, 13, 4104, 144, 0, 0, 2),
    _case(("ring", 128, 128, False), 2021, 3, 1032, 8208, 0),
    _case(("ring", 128, 128, True), 1000, 8, 1000, 16400, 8),
    _case(("persistent", 256, 256, False), 2021, 7, 4104, 528, 0, 3, 1),
    _case(("persistent", 256, 256, False), 4111, 13, 2056, 2064, 0),
    _case(("stream", 16, 16, False), 3, 1, 136, 2064, 0),
    _case(("stream", 16, 16, False), 75, 70, 264, 400, 0, 2, 2),
    _case(("stream", 16, 16, False), 37, 40, 72, 4112, 4),
]
