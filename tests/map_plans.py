"""Which plan the feature-map operators take for a map: the rules of
group_norm.cu, gn_cluster.cu and resize_map.cu over again, so that tests can
say which paths their sizes run.  Where a rule asks the GPU how many clusters
are resident, every plan that any answer could lead to is listed."""

SMS = 152
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def up(a, b):
    return -(-a // b)


def cluster_plans(shape, G, dtype, grad):
    """(cluster, vectors a thread, units, groups a slab, slabs) of every slab and cluster that hold an image; empty:
    the passes."""
    N, H, W, C = shape
    ve, Cg = 16 // SIZE[dtype], C // G
    base = next(b for b in range(1, ve + 1) if b * Cg % ve == 0)
    vecs = base * Cg // ve
    if C % ve or vecs > 32:
        return []
    plans = []
    for m in range(max(1, 8 // vecs), 0, -1):
        lv, gs = vecs * m, base * m
        if lv < 2 and gs < G:
            break
        # shared memory: kept vectors (dz as float32 beside x), a row a warp, five constants a channel, a sum a group
        slot = 256 * (16 + 4 * ve if grad else 16)
        fixed = 8 * 8 * lv * ve + up(20 * gs * Cg, 16) * 16 + 8 * gs
        rows, slabs = up(H * W, 8 * (32 // lv)), up(G, gs)
        for cl in range(1, 9):
            keep = up(rows, cl)
            if keep <= (112 * 1024 - fixed) // slot and up(rows, keep) == cl:
                plans.append((cl, keep, N * slabs, gs, slabs))
    return plans


def fewest_rounds(plan):
    """Units that a cluster takes at least: no more than two CTAs an SM are resident."""
    cl, _, units, _, _ = plan
    return up(units, 2 * SMS // cl)


def pass_plan(shape, ve, grad):
    """(chunks of an image, pixels a chunk, pixels a thread walks at most) of the pass kernels."""
    N, H, W, C = shape
    vecs, HW = C // ve, H * W
    lanes = 256 // min(vecs, 256)
    want = max(1, (3 if grad else 4) * SMS // (up(vecs, 256) * N))
    chunks = min(max(HW // (8 * lanes), 1), min(want, 4 * SMS))
    px = up(HW, chunks)
    return up(HW, px), px, up(px, lanes)


def wave_run(W, vecs, rows, images, slots, most):
    columns, best, run = up(W * vecs, 256), None, 0
    while most:
        cost = up(columns * images * up(rows, most), slots) * (most + 4)
        if best is None or cost < best:
            best, run = cost, most
        most //= 2
    return run


def resize_vector(C, dtype):
    return next(v for v in (16 // SIZE[dtype], 4, 2, 1) if C % v == 0)


def forward_run(N, geo, C, dtype):
    """Rows a thread of the resize walks."""
    H, W, OH, OW = geo
    return wave_run(OW, C // resize_vector(C, dtype), OH, N, 5 * SMS, 16)


def gradient_plan(N, geo, C, dtype, table=False):
    """(readers held, rows a thread walks, output rows ahead) of the resize's gradient."""
    H, W, OH, OW = geo
    v = resize_vector(C, dtype)
    if table:
        dtype, v = "f32", min(v, 4)
    readers = 4 if OW <= 2 * W else 6 if 2 * OW <= 5 * W else 8
    ctas = 4 if SIZE[dtype] == 4 and readers < 8 else 3
    run = wave_run(W, C // v, H, 1 if table else N, ctas * SMS, 32)
    return readers, run, 1 if run == 1 else (12 if ctas == 4 else 16) // readers


def likely_plan(shape, G, dtype, grad):
    """The plan of least estimated time if as many clusters were resident as have room.  One of single CTAs is then the
    plan that is taken: fewer resident clusters would make the others dearer only."""
    def cost(plan):
        cl, keep, *_ = plan
        barrier = 0.0 if cl == 1 else 0.3 * cl if grad else 0.6 + 0.1 * cl
        return fewest_rounds(plan) * ((2.3 + 0.62 * keep if grad else 2.8 + 0.35 * keep) + barrier)

    return min(cluster_plans(shape, G, dtype, grad), key=cost)


# ------------------------------------------------------------------ the cases
# Norms whose units are more than the clusters that are resident: single CTAs with a last slab of one group (every
# thread as many vectors, and unlike numbers of them), then clusters of several CTAs.
ROUNDS_ALONE = [(shape, 9, dtype, grad) for shape in ((256, 8, 8, 72), (256, 9, 7, 72)) for dtype in SIZE
                for grad in (False, True)]
ROUNDS_CLUSTERS = [((64, 64, 64, 64), 8, "bf16", False), ((64, 64, 64, 64), 8, "f32", False),
                   ((64, 40, 40, 64), 8, "bf16", True), ((64, 40, 40, 64), 8, "f16", True),
                   ((40, 56, 56, 64), 8, "f32", True)]
# Norms in passes with more chunks than one step of the join takes.
MANY_CHUNKS = [((1, 250, 255, 128), 32, "f32"), ((1, 250, 255, 128), 32, "bf16")]
# Resizes by what their gradient holds: 4, 6 and 8 readers, a reduction, single channels' longest runs.
RESIZES = [(8, (64, 64, 128, 128), 128), (8, (64, 60, 140, 147), 64), (8, (48, 48, 144, 144), 64),
           (8, (128, 128, 60, 61), 64), (304, (64, 85, 128, 170), 3)]
TABLE = (3, (64, 64, 100, 90), 512)
