"""Sizes of the adapters' tests that reach every kernel (m, k, n, rank, adapters), and
what the library says it takes for them."""
import re

import quantized_gemm_qg_amd as qg

# small: one launch.  The others: blocks of the rank x parts of k of the first product
# (among them 16, parts that are empty, a last group of fewer than four), row blocks x
# steps of the rank x one or more column chunks of the second, ranks that leave units
# of zeros, odd and even columns.
EVERY_KERNEL = [
    (2, 8, 64, 8, 1), (3, 8, 64, 24, 1), (1, 8, 67, 40, 1),
    (1, 8, 65, 136, 1), (1, 8424, 136, 16, 1), (1, 3360, 157, 40, 1), (1, 5648, 215, 24, 1), (6, 8, 72, 72, 1), (3990, 8, 67, 8, 42),
    (4318, 8, 80, 40, 9), (4, 552, 103, 72, 1), (1, 552, 75, 136, 1), (3, 2080, 103, 72, 1), (3, 2352, 66, 136, 1),
    (137, 544, 14942, 24, 1),
    (4152, 16, 1078, 8, 7), (3487, 112, 1281, 40, 1), (2925, 32, 1548, 72, 1), (549, 8, 11242, 8, 49),
    (1179, 16, 2642, 8, 63), (1047, 8, 7776, 24, 2), (3296, 16, 2319, 40, 1), (4799, 8, 1550, 72, 2), (4596, 8, 1352, 40, 35),
    (1234, 8, 2376, 16, 65), (1312, 16, 5688, 136, 5), (757, 8, 12714, 8, 35), (3070, 32, 3682, 40, 2), (4358, 8, 2646, 72, 2),
    (424, 888, 15769, 8, 11), (4523, 48, 2624, 16, 32), (1082, 584, 14895, 40, 2), (3843, 8, 4222, 136, 1), (3023, 16, 2060, 24, 70),
    (646, 152, 9528, 40, 19), (1357, 128, 12304, 72, 1), (1996, 32, 6808, 8, 53), (3331, 56, 4757, 40, 2), (2347, 16, 6775, 72, 2),
    (3999, 96, 1573, 72, 85)]


def taken(m, k, n, rank, adapters, y_type):
    """The kernels' numbers, e.g. {'NB': 1, 'splits': 3, 'RB': 2, 'SD': 1, 'chunks': 2} (one launch: NB alone)."""
    return {key: int(v) for key, v in re.findall(r"(\w+)=(\d+)", qg.describe_lora(m, k, n, adapters, rank, y_type))}
