"""The tilings that each dense product is built with (test support)."""
GLU, STORE, DGLU, WEIGHT, I8 = range(5)
PAIR = {GLU: [(2, 256), (2, 224), (2, 192), (2, 160), (2, 128)],
        STORE: [(2, 256), (2, 224), (2, 192), (2, 160), (1, 256), (1, 192), (1, 160), (1, 128)],
        DGLU: [(1, 256), (1, 224), (1, 192), (1, 160), (1, 128)],
        WEIGHT: [(2, 256), (1, 256)],
        I8: [(1, 256), (1, 224), (1, 192), (1, 160), (1, 128)]}
SPLIT = [(nt, split) for nt in (16, 32, 48, 64, 128) for split in (1, 2, 4, 5, 6, 8)]
