"""One small product for every form that the library's choice can take on 148 SMs:
(operand type, rows per expert, N, K, (CTAs per tile, rows per tile, CTAs along K),
pieces per tile of the last turn). Used by the GPU tests, and checked against the
choice itself without a GPU."""


def spread(rows, experts):
    """Uneven groups, the first of them empty where there is more than one."""
    if experts == 1:
        return [rows]
    counts = [0] + [1 + (3 * i) % 7 for i in range(experts - 1)]
    counts[-1] += rows - sum(counts)
    return counts


FORMS = [
    ("bf16", spread(1, 1), 96, 48, (1, 16, 1), 1),
    ("int8", spread(5, 2), 130, 96, (1, 16, 1), 1),
    ("bf16", [0, 1, 0, 3] + [1] * 10 + [0, 0], 281, 896, (1, 16, 2), 1),
    ("int8", [0, 1, 0, 3] + [1] * 10 + [0, 0], 281, 1744, (1, 16, 2), 1),
    ("bf16", spread(3, 1), 97, 1040, (1, 16, 4), 1),
    ("int8", spread(3, 1), 97, 2064, (1, 16, 4), 1),
    ("bf16", spread(273, 16), 388, 64, (1, 32, 1), 1),
    ("int8", spread(273, 16), 388, 64, (1, 32, 1), 1),
    ("bf16", spread(290, 16), 264, 1328, (1, 32, 2), 1),
    ("int8", spread(290, 16), 266, 2640, (1, 32, 2), 1),
    ("bf16", spread(71, 4), 532, 1024, (1, 32, 4), 1),
    ("int8", spread(71, 4), 532, 2064, (1, 32, 4), 1),
    ("bf16", spread(257, 8), 1026, 64, (1, 64, 1), 1),
    ("int8", spread(257, 8), 1026, 64, (1, 64, 1), 1),
    ("bf16", spread(561, 16), 262, 2128, (1, 64, 2), 1),
    ("int8", spread(561, 16), 262, 4208, (1, 64, 2), 1),
    ("bf16", spread(551, 4), 136, 1328, (1, 64, 4), 1),
    ("int8", spread(573, 4), 131, 2576, (1, 64, 4), 1),
    ("bf16", spread(259, 4), 2099, 64, (1, 128, 1), 1),
    ("int8", spread(259, 4), 2099, 64, (1, 128, 1), 1),
    ("bf16", spread(1116, 16), 263, 2576, (1, 128, 2), 1),
    ("int8", spread(1113, 16), 263, 4816, (1, 128, 2), 1),
    ("bf16", spread(533, 8), 277, 1872, (1, 128, 4), 1),
    ("int8", spread(1027, 8), 139, 4112, (1, 128, 4), 1),
    ("bf16", spread(2104, 3), 130, 272, (2, 64, 1), None),
    ("int8", spread(2281, 4), 129, 528, (2, 64, 1), None),
    ("bf16", spread(4163, 8), 130, 144, (2, 96, 1), None),
    ("int8", spread(1737, 16), 133, 704, (2, 96, 1), None),
    ("bf16", [2, 515], 4719, 64, (2, 128, 1), 1),
    ("int8", [5, 10, 1027, 6], 2345, 64, (2, 128, 1), 1),
    ("bf16", [221, 315], 4761, 64, (2, 128, 1), 2),
    ("int8", [184, 548, 65], 3132, 64, (2, 128, 1), 2),
    ("bf16", spread(2796, 8), 257, 144, (2, 160, 1), None),
    ("int8", spread(5181, 16), 514, 48, (2, 160, 1), None),
    ("bf16", spread(4797, 4), 387, 48, (2, 192, 1), None),
    ("int8", spread(3483, 3), 527, 48, (2, 192, 1), None),
    ("bf16", spread(3628, 4), 526, 48, (2, 224, 1), None),
    ("int8", spread(3789, 4), 532, 48, (2, 224, 1), None),
    ("bf16", [303, 7, 2, 7], 4973, 64, (2, 256, 1), 2),     # pieces of the narrow tiles have no rows
    ("int8", [3, 265, 19, 6], 4800, 64, (2, 256, 1), 2),
    ("bf16", [135, 101, 98, 411], 4148, 64, (2, 256, 1), 4),
    ("int8", [2062, 3652, 140], 527, 64, (2, 256, 1), 4),
    ("bf16", [2, 6, 1, 2], 4932, 128, (2, 256, 1), 4),
    ("int8", [1, 1, 4, 2], 4863, 64, (2, 256, 1), 4),
    ("bf16", [4095], 4096, 64, (2, 256, 1), 2),
]
