"""Plain 64-bit definitions of the paged 8-bit cache's operators (numpy, no GPU code).

Written from the definitions in include/oasis.h; only tests use it.  A cache is a
dict: kv uint8 [n_pages][Hkv][2][16][128], scale float64 [n_pages][Hkv][2], table int
[B][nb_max].
"""
import numpy as np

BS, D = 16, 128
E_LOW, E_HIGH = -60, 119


def _e4m3_values():
    v = np.empty(256)
    for b in range(256):
        s, e, m = -1.0 if b & 0x80 else 1.0, (b >> 3) & 15, b & 7
        v[b] = np.nan if b & 0x7f == 0x7f else s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


E4M3 = _e4m3_values()
_POS = E4M3[:0x7f]  # 0 .. 448, ascending with the byte


def e4m3_bytes(x):
    """Bytes of the nearest e4m3 values, ties to the even mantissa, saturating at 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 0x7e)  # the first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    b = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), 0x7f, b | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def exponent(amax):
    """The least e in [E_LOW, E_HIGH] with amax <= 448 * 2^e (E_HIGH if none)."""
    for e in range(E_LOW, E_HIGH):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_HIGH


def extend_tables(old, new, free, n_free, table, n_rows, n_pages):
    """(lens, n_free, row_start, slot_map, table, error bits)."""
    B, nb_max = table.shape
    table, slots, lens, start, bits = table.copy(), np.full(n_rows, -1, np.int64), [], [], 0
    if not 0 <= n_free <= n_pages:
        bits |= 8
        n_free = min(max(n_free, 0), n_pages)
    row = need_before = left_out = 0
    left = n_free
    for b in range(B):
        o, n = int(old[b]), int(new[b])
        bad = o < 0 or n < o or n > nb_max * BS
        start.append(min(row, n_rows))
        if bad:
            bits |= 8
            lens.append(o)
            continue
        held = -(-o // BS)
        need = -(-n // BS) - held
        no_page = need > 0 and need_before + need > n_free
        no_room = row + n - o > n_rows
        bits |= (4 if no_page else 0) | (8 if no_room else 0)
        if not (no_page or no_room):
            for i in range(need):
                p = int(free[n_free - 1 - (need_before + i)])
                if not 0 <= p < n_pages:
                    bits |= 1
                    p = -1
                table[b, held + i] = p
            left -= need
            for t in range(o, n):
                p = int(table[b, t // BS])
                if 0 <= p < n_pages:
                    slots[row + t - o] = p * BS + t % BS
                else:
                    bits |= 1
        lens.append(o if no_page or no_room else n)
        row += n - o
        need_before += need
    start.append(min(row, n_rows))
    return np.array(lens), left, np.array(start), slots, table, bits


def release_tables(lens, keep, table, free, n_free, n_pages):
    """(free list, n_free, error bits)."""
    free, bits = free.copy(), 0
    for b in range(table.shape[0]):
        if not 0 <= keep[b] <= lens[b] <= table.shape[1] * BS:
            bits |= 8
            continue
        for x in range(-(-int(keep[b]) // BS), -(-int(lens[b]) // BS)):
            p = int(table[b, x])
            if not 0 <= p < n_pages:
                p = -1
                bits |= 1
            if n_free < n_pages:
                free[n_free] = p
                n_free += 1
            else:
                bits |= 4
    return free, n_free, bits


def store(kv, scale, k, v, slots):
    """k, v float64 [rows][Hkv][128]; returns (kv, scale, error bits) after the call."""
    kv, scale, bits = kv.copy(), scale.copy(), 0
    n_slots, i, n = kv.shape[0] * BS, 0, len(slots)
    while i < n:
        s = int(slots[i])
        if not 0 <= s < n_slots:
            bits |= 2 if s != -1 else 0
            i += 1
            continue
        if i > 0 and 0 <= slots[i - 1] and slots[i - 1] // BS == s // BS:  # a broken run
            bits |= 8 if s != slots[i - 1] + 1 else 0
            i += 1
            continue
        j = i + 1
        while j < n and slots[j] == s + j - i and (s + j - i) // BS == s // BS:
            j += 1
        p, pos = divmod(s, BS)
        for h in range(kv.shape[1]):
            for w, x in enumerate((k, v)):
                rows = x[i:j, h]
                e = exponent(np.abs(rows).max())
                if pos:
                    old = int(np.clip(np.round(np.log2(scale[p, h, w])), E_LOW, E_HIGH))
                    if e > old:
                        kv[p, h, w, :pos] = e4m3_bytes(E4M3[kv[p, h, w, :pos]] * 2.0 ** (old - e))
                    e = max(e, old)
                scale[p, h, w] = 2.0 ** e
                kv[p, h, w, pos:pos + j - i] = e4m3_bytes(rows * 2.0 ** -e)
        i = j
    return kv, scale, bits


def _softmax_rows(q, k, v, scale):
    """q [rows][D], k, v [tokens][D]: (outputs, sum p |v|, largest |q||k| * scale, sum of exp(s - max))."""
    s = q @ k.T * scale
    p = np.exp(s - s.max(axis=-1, keepdims=True))
    total = p.sum(axis=-1, keepdims=True)
    size = np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max() * scale
    return p @ v / total, p @ np.abs(v) / total, size, total


def decode(q, kv, scale, table, ctx, softmax_scale, sel=None, nsel=None):
    """(out, sum p |v|, |q||k| scale per pair, error of weights below fp16's normal range per pair)."""
    B, Hq, _ = q.shape
    Hkv, n_pages = kv.shape[1], kv.shape[0]
    G = Hq // Hkv
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    size, tiny = np.zeros((B, Hq, 1)), np.zeros((B, Hq, 1))
    for b in range(B):
        n = min(max(int(ctx[b]), 0), table.shape[1] * BS)
        for h in range(Hkv):
            nb = -(-n // BS)
            blocks = range(nb) if sel is None else [int(x) for x in sel[b, h, : min(max(int(nsel[b, h]), 0), sel.shape[2])]]
            ks, vs = [], []
            for x in blocks:
                if not 0 <= x < nb or not 0 <= table[b, x] < n_pages:
                    continue
                p, m = int(table[b, x]), min(BS, n - x * BS)
                ks.append(E4M3[kv[p, h, 0, :m]] * scale[p, h, 0])
                vs.append(E4M3[kv[p, h, 1, :m]] * scale[p, h, 1])
            if not ks:
                continue
            ks, vs, r = np.concatenate(ks), np.concatenate(vs), slice(h * G, h * G + G)
            out[b, r], mass[b, r], size[b, r], total = _softmax_rows(q[b, r], ks, vs, softmax_scale)
            tiny[b, r] = len(ks) * np.abs(vs).max() / total
    return out, mass, size, tiny


def prompt(q, k, v, row_start, softmax_scale):
    """(out, sum p |v|, |q||k| scale); rows of no sequence are zero."""
    G = q.shape[1] // k.shape[1]
    out, mass, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2] + (1,))
    for a, z in zip(row_start[:-1], row_start[1:]):
        for i in range(int(a), int(z)):
            for h in range(k.shape[1]):
                r = slice(h * G, h * G + G)
                out[i, r], mass[i, r], size[i, r], _ = _softmax_rows(q[i, r], k[a:i + 1, h], v[a:i + 1, h], softmax_scale)
    return out, mass, size
