"""How the backward of the norms around a block (csrc/block_norm.hip) adds its columns' sums:
the launch as sizes decide it, for bars and for choosing sizes.  A CPU test holds it to
the library's workspace."""


def backward_plan(rows, width):
    """(workgroups, rows of a workgroup at a time, times that it takes so many)."""
    tpr = 16
    while 8 * tpr < width and tpr < 1024:
        tpr *= 2
    if width <= 8192:
        tpr = min(tpr, 512)
    threads, waves = (768, 3) if tpr <= 128 else (tpr, {256: 3, 512: 2, 1024: 4}[tpr])
    per = threads // tpr
    need, most = -(-rows // per), 256 * (waves * 256 // threads)
    times = -(-need // most)
    if per == 1:
        times = max(times, min(4, -(-need // 128)))
    blocks = -(-need // times)
    return blocks, per, -(-need // blocks)


def column_depth(rows, width):
    """Additions that a value goes through at most, from a thread's first row to the total: its
    thread's other rows, the workgroup's other rows of a time, the partial rows of a
    group of 64 apart, eight groups, and eight of those."""
    blocks, per, times = backward_plan(rows, width)
    return times + per + -(-blocks // 64) + 8 + 8
