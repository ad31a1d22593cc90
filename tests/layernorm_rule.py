"""The rule by which the layer norm's launches are chosen (csrc/zero_layernorm.cuh,
zero_layernorm.cu, zero_layernorm_backward.cu), restated, so that a test can say
which kernel and how many row groups its sizes reach."""

SMEM, MOST_THREADS, F32 = 216 * 1024, 512, "f32"


def _words(t):
    return 2 if t == F32 else 1


def rows_shape(rows, cols, nv, words, vectors, sms):
    """(threads a row, rows a block, blocks), or None: the row does not fit."""
    units = -(-cols // 8)
    t = -(-units // (32 * nv)) * 32
    if t > MOST_THREADS:
        return None
    g = min(-(-rows // sms), MOST_THREADS // t)
    stage, fixed = (words * nv * 32 + 3) * 16 * (t // 32), vectors * 16 * units
    while g > 1 and 2 * stage * g + fixed > SMEM:
        g -= 1
    if 2 * stage * g + fixed > SMEM:
        return None
    return t, g, min(-(-rows // g), sms)


def _either(rows, cols, words, vectors, sms):
    two, four = (rows_shape(rows, cols, nv, words, vectors, sms) for nv in (2, 4))
    threads = lambda s: s[0] * s[1] if s else 0
    return (4, four) if cols > 512 and threads(four) >= threads(two) else (2, two)


def kernel(backward, rows, cols, xt, rt, wt, aligned, sms):
    """(template, groups of rows a block, blocks, rule): template is
    (direction, x's type, the residual's, units a lane or "long", weights kept
    packed, rows that start anywhere); rule says how the units were chosen."""
    words = _words(xt) + (2 if backward else 1) * _words(rt)
    vectors, packed_vectors = (2, 1) if backward else (4, 2)
    nv, s = _either(rows, cols, words, vectors, sms)
    rule = "plain"
    if backward and not aligned and nv == 4:
        two = rows_shape(rows, cols, 2, words, vectors, sms)
        if two and s and two[0] * two[1] * 5 > s[0] * s[1] * 4:
            nv, s, rule = 2, two, "two for their threads"
    packed = s is None and xt != F32 and wt == xt
    if packed:
        nv, s = 4, rows_shape(rows, cols, 4, words, packed_vectors, sms)
    if s is None:
        return ("backward" if backward else "forward", xt, rt, "long", False, not aligned), 1, 0, "long"
    return ("backward" if backward else "forward", xt, rt, nv, packed, not aligned), s[1], s[2], rule
